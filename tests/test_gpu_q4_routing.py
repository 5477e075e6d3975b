"""Routing of the 4-bit decode where its logits are unusual: of any size, and not finite.  The summaries are set by
hand so that every logit is a float32 number and no rounding happens before the thresholds."""
import numpy as np
import pytest
import torch

import adaptive_sparse_hierarchical_b200 as D

pytestmark = pytest.mark.gpu

# one block that attends too, one block per row, the whole GPU, rows beyond a block's registers
FORMS = [(64, 32, 4), (300, 32, 4), (1000, 32, 16), (20000, 16, 2)]


def _weights(x, alpha):
    """Entmax weights of x [.., T] (float64), by bisection on the differences to the maximum."""
    x = x - x.max(-1, keepdims=True)
    p = 1 / (alpha - 1)
    lo, hi = -np.ones(x.shape[:-1] + (1,)), np.zeros(x.shape[:-1] + (1,))
    for _ in range(80):
        mid = (lo + hi) / 2
        over = (np.maximum(x - mid, 0) ** p).sum(-1, keepdims=True) > 1
        lo, hi = np.where(over, mid, lo), np.where(over, hi, mid)
    u = np.maximum(x - (lo + hi) / 2, 0)
    return u ** p, u


def _routes(st, b):
    hkv, T = st.kbar.shape[1], st.T
    rt = [torch.zeros(b, hkv, dtype=torch.int32, device="cuda"), torch.full((b, hkv, T), -1, dtype=torch.int32, device="cuda"),
          torch.zeros(b, hkv, T, device="cuda"), torch.full((b, hkv, (T + 31) // 32), -1, dtype=torch.int32, device="cuda")]
    st.route = D.route_out(*rt)
    return rt


def _cache(T, B, g, alpha, gamma, d=64, hkv=2):
    """An empty cache of T chunks on one page that every slot names."""
    cap = T * B + 5
    slots = -(-cap // B)
    return D.Q4DecodeState(1, cap, g * hkv, hkv, d, chunk=B, alpha=alpha, gamma=gamma, page_size=B, num_pages=1,
                           page_table=torch.zeros(1, slots, dtype=torch.int32))


@pytest.mark.parametrize("T,B,g", FORMS)
@pytest.mark.parametrize("alpha", [1.5, 2.0])
@pytest.mark.parametrize("top", [0.0, 2.0 ** 10, -2.0 ** 17, 2.0 ** 17, 2.0 ** 24, 2.0 ** 40, -2.0 ** 60])
def test_logits_of_any_size(T, B, g, alpha, top):
    """The routes depend on the differences to the largest logit only: rows top - k 2^-6 (or as fine as float32 has
    them there) against entmax in 64 bits."""
    rng = np.random.default_rng(int(abs(top)) % 1000 + T + g)
    hkv, d = 2, 64
    st = _cache(T, B, g, alpha, 16.0 if alpha == 1.5 else 8.0)   # (alpha - 1) gamma / sqrt(d) = 1
    unit = max(2.0 ** -6, abs(top) * 2.0 ** -23)
    # of each head: a few chunks at the top, some near it, the others below
    steps = rng.integers(0, 64, (hkv, g, T)) * np.where(rng.random((hkv, g, T)) < 30 / T, 1, 3) + 20
    steps[:, :, rng.permutation(T)[:3]] = 0
    low = -steps * unit
    kbar = torch.zeros(hkv, T, d, dtype=torch.float64)
    kbar[:, :, 0] = 1.0 if top >= 0 else -1.0
    kbar[:, :, 1:1 + g] = torch.from_numpy(low).transpose(1, 2)
    q = torch.zeros(hkv, g, d, dtype=torch.float64)
    q[:, :, 0] = abs(top)
    for h in range(g):
        q[:, h, 1 + h] = 1.0
    st.kbar[0].copy_(kbar)
    st.seqlens.fill_(T * B + 3)
    rt = _routes(st, 1)
    st.decode(q.view(1, hkv * g, d).bfloat16().cuda())
    counts, idx, bias, mask = (t[0].cpu().numpy() for t in rt)
    w, u = _weights(top + low, alpha)
    w = w.mean(1)                                            # [hkv, T]
    # The threshold: the mass f is a sum of at most `inside` products, rounded by 2^-24 a step, and its slope is at
    # least 1 (alpha 2: the size of the support; alpha 1.5: twice the sum of u, whose squares sum to 1), the solve
    # stops within 1e-6 of mass or 2e-7 of t.
    inside = (u > 0).sum(-1).max()
    dt = (inside + 32) * 2.0 ** -24 + 1.2e-6
    for r in range(hkv):
        # a chunk is certain if some head's margin is beyond dt, or all heads' entries are that far outside
        x = top + low[r]
        thr = (x.max(-1, keepdims=True) - x).astype(float)   # distance below the maximum
        tau = np.array([(thr[h] + u[r, h])[u[r, h] > 0].min() for h in range(g)])[:, None]
        sure_in, maybe = (tau - thr > dt).any(0), (tau - thr > -dt).any(0)
        got = np.zeros(T, bool)
        got[idx[r, :counts[r]]] = True
        assert (np.diff(idx[r, :counts[r]]) > 0).all()
        assert not (sure_in & ~got).any() and not (got & ~maybe).any(), (r, sure_in.sum(), got.sum())
        bits = ((mask[r].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1)[:T] != 0
        assert np.array_equal(bits, got)
        if not np.array_equal(got, w[r] > 0):
            continue
        # log w: a head's weight u^p is off by p u^(p-1) dt and two roundings, the mean over heads by as much more
        p = 1 / (alpha - 1)
        dw = (p * np.where(u[r] > 0, u[r], 0) ** (p - 1) * dt * (u[r] > 0) + 4 * 2.0 ** -24 * u[r] ** p).mean(0) + g * 2.0 ** -24 * w[r]
        lw, dl = np.log(w[r][got]), dw[got] / w[r][got]
        if dl.max() > 0.1:
            continue
        # (the device's logarithm is within 2^-21.4 absolutely, and the mean of n of them within n roundings)
        tol = 1.2 * (dl + dl.mean()) + 2 * 2.0 ** -21 + (got.sum() + 32) * 2.0 ** -24 * np.abs(lw).max()
        assert (np.abs(bias[r, :counts[r]] - (lw - lw.mean())) <= tol).all(), r


@pytest.mark.parametrize("T,B,g", FORMS)
@pytest.mark.parametrize("alpha", [1.5, 2.0, 1.25])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_keys_that_are_not_numbers(T, B, g, alpha, bad):
    """A completed chunk whose summary is not finite reaches the outputs of its KV head, as the chunk's keys do
    without routing; other heads and sequences are as without it."""
    rng = np.random.default_rng(T)
    d, hkv, slots = 64, 2, T + 1
    st = D.Q4DecodeState(2, T * B + 5, g * hkv, hkv, d, chunk=B, alpha=alpha, gamma=3.0, page_size=B, num_pages=2,
                         page_table=torch.arange(2, dtype=torch.int32).view(2, 1).repeat(1, slots))
    st.kbar.copy_(torch.from_numpy(rng.standard_normal((2, hkv, T, d))))
    for t in (st.k_codes, st.v_codes):
        t.random_(0, 256)
    st.k_scales.fill_(0x38)
    st.v_scales.fill_(0x38)
    st.seqlens.copy_(torch.tensor([T * B + 3, T * B - 1], dtype=torch.int32))
    q = torch.from_numpy(rng.standard_normal((2, g * hkv, d))).bfloat16().cuda()
    clean = st.decode(q).clone()
    assert torch.isfinite(clean).all()
    st.kbar[0, 1, T - 2, 7] = bad
    st.kbar[0, 1, T - 2, 9] = -bad
    rt = _routes(st, 2)
    o = st.decode(q).clone()
    assert torch.isnan(o[0, g:]).all()
    assert torch.equal(o[0, :g], clean[0, :g]) and torch.equal(o[1], clean[1])
    n = int(rt[0][0, 1])
    assert T - 2 in rt[1][0, 1, :n].tolist() and torch.isnan(rt[2][0, 1, :n]).all()
    # a query that is not a number stays in its head
    st.kbar[0, 1, T - 2, 7] = st.kbar[0, 1, T - 2, 9] = 0.0
    q[1, 1, 3] = bad
    o = st.decode(q)
    assert torch.isnan(o[1, 1]).all() and torch.isfinite(o[1, 0]).all() and torch.isfinite(o[1, 2:]).all()
    assert torch.isfinite(o[0]).all()
