"""The bound on a page score's error (csrc/score_error.h) against what two 16-bit terms leave of a folded query."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def pieces(tmp_path_factory):
    exe = tmp_path_factory.mktemp("score_error") / "score_error_example"
    r = subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "paged_decode_attention_cache_gb300", "csrc"),
                        os.path.join(ROOT, "tests", "c", "score_error_example.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60).stdout.split("\n")
    return {torch.bfloat16: [float(x) for x in lines[0].split()], torch.float16: [float(x) for x in lines[1].split()]}


def weights(dtype):
    """Folded queries, sums of up to 8 numbers of `dtype`, and among them those whose terms leave most; fp16's scaled to at most 2^15."""
    g = torch.Generator().manual_seed(0)
    w = (torch.randn(8, 1 << 20, generator=g) * 2.0 ** torch.randint(-18, 1, (8, 1 << 20), generator=g)).to(dtype).abs().float()
    w = w.cumsum(0).flatten()
    most = torch.tensor([1.0 + 2.0 ** -8 - 2.0 ** -16 + 2.0 ** -17 * (1 - 2.0 ** -6)])
    if dtype == torch.float16:
        w, most = w * 2.0 ** 14 / w.max(), torch.tensor([2.0 ** -9 + 2.0 ** -25 * (1 - 2.0 ** -6)])
    return torch.cat([w, most])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_two_terms(pieces, dtype):
    terms, others, short, bound = pieces[dtype]
    w = weights(dtype).double()
    first = w.to(dtype).double()
    left = (w - first - (w - first).to(dtype).double()).abs() / (w if dtype == torch.bfloat16 else w.clamp(min=2.0 ** -7))
    worst = float(left.max())
    assert terms / 1.02 < worst <= terms
    assert (worst + others) <= bound * (1 - short)
