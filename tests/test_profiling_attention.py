"""Profiles of the attention layer: kernel names, and the digest that tells when the
sources have changed since."""

import glob
import os
import re

import pytest

from gated_delta_rule_54_amd import profiling

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = "gdr::(anonymous namespace)::"


@pytest.mark.parametrize("name,want", [
    (f"void {G}attn_fwd_kernel<unsigned short, unsigned short, 128, 2, true>(gdr::AttnArgs)", "attention"),
    (f"void {G}attn_dq_kernel<unsigned short, float, 64, 3, false>(gdr::AttnArgs)", "attention_dq"),
    (f"void {G}attn_dkv_kernel<float, float, 256, 3>(gdr::AttnArgs, {G}Parts)", "attention_dkv"),
    (f"void {G}attn_join_kernel<float, float, 256>(gdr::AttnArgs, {G}Parts)", "attention_join"),
    (f"void {G}cache_attn_kernel<unsigned short, float, 64>(gdr::CacheAttnArgs, int, int, bool, int)", "cache_attention"),
    (f"void {G}cache_join_kernel<float>(gdr::CacheAttnArgs, int)", "cache_join"),
    (f"void {G}rotary_kernel<unsigned short, float>(gdr::RotArgs, int)", "rotary"),
    (f"void {G}decode_kernel<float>(int)", "decode"),
])
def test_label(name, want):
    assert profiling.label(name) == want


def test_digest_follows_its_sources_alone(tmp_path, monkeypatch):
    src = os.path.join(os.path.dirname(profiling.__file__), "csrc")
    (tmp_path / "csrc").mkdir()
    for f in os.listdir(src):
        (tmp_path / "csrc" / f).write_bytes(open(os.path.join(src, f), "rb").read())
    before = [profiling.src_digest(), profiling.src_digest(True), profiling.src_digest(attention=True)]
    assert len(set(before)) == 3
    monkeypatch.setattr(profiling, "_HERE", str(tmp_path))

    def changed(name):
        p = tmp_path / "csrc" / name
        old = p.read_bytes()
        p.write_bytes(old + b"\n")
        now = [profiling.src_digest(), profiling.src_digest(True), profiling.src_digest(attention=True)]
        p.write_bytes(old)
        return [a != b for a, b in zip(now, before)]

    for f in ("gdr_attn.hip", "gdr_attn.h", "gdr_cache.hip", "gdr_rotary.hip"):
        assert changed(f) == [False, False, True]
    assert changed("gdr_norm.hip") == [False, True, False] and changed("gdr_seq.hip") == [True, False, False]
    assert changed("gdr_device.h") == [True, True, True]


def test_stored_profiles_carry_a_digest():
    found = glob.glob(os.path.join(ROOT, "profiles", "*attention_layer*.md"))
    assert found
    for p in found:
        assert re.search(r"^Kernel sources digest: `[0-9a-f]{16}`$", open(p).read(), re.M), p
