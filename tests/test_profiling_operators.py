"""Profiles of the operators beside the rule: kernel names, and the digest that
tells when the sources have changed since."""

import glob
import os
import re

import pytest

from gated_delta_rule_54_amd import profiling

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = "gdr::(anonymous namespace)::"


@pytest.mark.parametrize("name,want", [
    (f"void {G}lin_chunk_kernel<{G}OpB<64>, 128, {G}Job<2, false, false, false>, {G}Job<2, false, false, false> >"
     "(gdr::LinChains)", "linear_chunks"),
    (f"void {G}lin_chunk_kernel<{G}OpB<64>, 128, {G}Job<3, true, true, false>, {G}Job<2, false, false, false> >"
     "(gdr::LinChains)", "linear_chunks_vjp"),
    (f"void {G}lin_chunk_kernel<{G}OpB<64>, 128, {G}Job<3, true, false, true>, {G}Job<2, false, false, false> >"
     "(gdr::LinChains)", "linear_chunks_vjp_add"),
    (f"void {G}lin_segment_kernel<{G}OpF, 64>(gdr::LinChains)", "linear_segments"),
    (f"{G}lin_dg_kernel(float const*)", "linear_dg"), (f"{G}lin_dg_head_kernel(double const*)", None),
    (f"void {G}norm_bwd_kernel<unsigned short, float, 16>(gdr::NormArgs, int)", "norm_bwd"),
])
def test_label(name, want):
    assert profiling.label(name) == want


def test_digests_follow_their_sources(tmp_path, monkeypatch):
    src = os.path.join(os.path.dirname(profiling.__file__), "csrc")
    (tmp_path / "csrc").mkdir()
    for f in os.listdir(src):
        (tmp_path / "csrc" / f).write_bytes(open(os.path.join(src, f), "rb").read())
    before = profiling.src_digest(), profiling.src_digest(True)
    monkeypatch.setattr(profiling, "_HERE", str(tmp_path))
    assert (profiling.src_digest(), profiling.src_digest(True)) == before

    def changed(name):
        p = tmp_path / "csrc" / name
        old = p.read_bytes()
        p.write_bytes(old + b"\n")
        now = profiling.src_digest() != before[0], profiling.src_digest(True) != before[1]
        p.write_bytes(old)
        return now

    assert changed("gdr_linear_chunk.hip") == changed("gdr_norm.h") == (False, True)
    assert changed("gdr_chunk16.hip") == (True, False) and changed("gdr_device.h") == (True, True)


def test_stored_profiles_carry_a_digest():
    found = glob.glob(os.path.join(ROOT, "profiles", "*linear*.md"))
    assert found
    for p in found:
        assert re.search(r"^Kernel sources digest: `[0-9a-f]{16}`$", open(p).read(), re.M), p
