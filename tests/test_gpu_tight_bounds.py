"""The attention's error bounds as its arithmetic gives them, where the other tests hold it to wider ones: 8-bit caches
with bf16 outputs (the weights are split in two fp16 halves for every output type), and the scored call over K8/V4 caches."""
import numpy as np
import pytest
import torch

from paged_decode_attention_cache_gb300 import ops
from tests import blocks_reference as R
from tests.helpers import GuardedOut
from tests.test_gpu_blocks import CTX, attend, close, filled, rows, want_attention
from tests.test_gpu_scored import make, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_decode_attention_cache_gb300 import build
    build.build()
    ops.lib()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("schedule", ["single", "split", "balanced", "noalloc", "scored"])
@pytest.mark.parametrize("kind,H,Hkv,D,ql", [("i8", 8, 2, 128, 1), ("e4m3", 16, 2, 64, 1), ("i8", 8, 2, 128, 4), ("e4m3", 8, 8, 64, 16)])
def test_bf16_outputs_of_8_bit_caches(schedule, kind, H, Hkv, D, ql):
    # bf16's half step is the relative term; the weights' 2^-22 the absolute one
    rng = np.random.default_rng(61 + H + D + ql)
    ctx = [c if c == 0 else max(c, ql) for c in CTX]
    st, seqs = filled(rng, kind, ctx, Hkv, D)
    seqs.q_len = ql
    q, qr = rows(rng, len(ctx) * ql, H, D, "bf16", 1.0)
    g = GuardedOut(q.shape, torch.bfloat16, "cuda")
    more = {}
    if schedule == "scored":
        more = dict(cap=20.0)
        ops.pkv_paged_attention_scored(g.out, q, D ** -0.5, st.cache, seqs, ops.Scores(20.0), ops.balanced_workspace(len(ctx), Hkv, D),
                                       st.err)
    else:
        attend(st, seqs, q, g.out, schedule, D ** -0.5)
    g.check()
    assert int(st.err.item()) == 0
    close(g.out, *want_attention(st, qr, ctx, ql, D ** -0.5, **more), torch.bfloat16, p_bits=22)


@pytest.mark.parametrize("dt,H,Hkv,D,ql", [("bf16", 8, 2, 128, 1), ("f16", 8, 1, 64, 2), ("f16", 4, 4, 64, 1), ("bf16", 8, 2, 128, 4)])
@pytest.mark.parametrize("what", ["plain", "cap", "bias"])
def test_scored_k8v4(what, dt, H, Hkv, D, ql):
    """The scores: codes + 1152 times q, exact products, in fp32 sums from which 1152 sum(q) is taken: the magnitudes that
    are rounded are 1279 k_scale sum|q| scale, off by at most 2^-19 of it (as in blocks_reference.tolerance), twice in a
    weight.  The weights: rounded to fp16 (2^-11, and 2^-25 below its normal numbers), times the V scale rounded again
    (likewise), against the zero point once; the sum of weights is fp32's.  A V code is at most 15."""
    rng = np.random.default_rng(62 + H + D + ql)
    ctx = [c if c == 0 else max(c, ql) for c in CTX]
    cache, tables, k, v = make(rng, "k8v4", ctx, Hkv, D, [np.zeros(c, bool) for c in ctx], dt)
    B, scale = len(ctx), D ** -0.5
    q, qr = rows(rng, B * ql, H, D, dt, 0.5)
    q, qr = q * 0.25, (q * 0.25).double().cpu().numpy()
    cap, slopes = (2.0 if what == "cap" else 0.0), (slopes_of(H) if what == "bias" else None)
    seqs = ops.Seqs(torch.from_numpy(tables).cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), ql)
    scores = ops.Scores(cap, None if slopes is None else torch.tensor(slopes, device="cuda"))
    g = GuardedOut(q.shape, torch.float32, "cuda")
    ops.pkv_paged_attention_scored(g.out, q, scale, cache, seqs, scores, ops.balanced_workspace(B, Hkv, D))
    g.check()
    want, biggest = R.attention(qr, k, v, ctx, ql, scale, 0, cap, slopes)
    finite = lambda t: t.float()[torch.isfinite(t)].abs().max().item()  # noqa: E731  (blocks without a token hold NaN)
    ks, vs, vz = finite(cache.k_scale), finite(cache.v_scale), finite(cache.v_zero)
    vmax = max(np.abs(x).max() for x in v if x.size)
    score = max(biggest, 1279 * ks * np.abs(qr).sum(-1).max() * scale)
    small = max(ctx) * 2.0 ** -25 * (15 + 15 * vs + vz)
    allowed = vmax * (2 * 2.0 ** -19 * (score + 1) + 2.0 ** -20) + 2.0 ** -11 * (2 * 15 * vs + vz) + small
    got = g.out.double().cpu().numpy()
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    print(f"{what} {dt} {H} {Hkv} {D} {ql}: max err {err.max():.2e}, allowed {allowed:.2e}")
    assert (err <= allowed + 2.0 ** -24 * np.abs(want)).all(), f"max err {err.max():.3e}, allowed {allowed:.3e}"
