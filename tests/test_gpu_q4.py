"""The 4-bit paged cache on the GPU (dash_append_q4 / dash_load_q4 / dash_decode_q4) against the float64
definitions of q4_ref.py: codes and scales bit for bit, values read back exactly, summaries and outputs
within bounds counted from the roundings."""
import math

import numpy as np
import pytest
import torch

import oracle
import adaptive_sparse_hierarchical_b200 as D
from adaptive_sparse_hierarchical_b200 import inputs

import q4_ref as R
from parity import bias_tolerance, check_routes

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(torch.bfloat16)


def _state(rng, b, cap, hq, hkv, d, *, chunk, page, alpha=1.5, gamma=4.0, k_exp=0, v_exp=0, slack=3):
    slots = -(-cap // page)
    pages = b * slots + slack
    table = torch.from_numpy(rng.permutation(pages)[: b * slots].reshape(b, slots).astype(np.int32))
    qbar = torch.from_numpy(rng.standard_normal((hkv, d)).astype(np.float32) * 0.3).cuda()
    return D.Q4DecodeState(b, cap, hq, hkv, d, chunk=chunk, alpha=alpha, gamma=gamma, page_size=page, num_pages=pages,
                           page_table=table, k_exp=k_exp, v_exp=v_exp, qbar=qbar)


def _gather(st, name, i, n):
    """Rows 0..n-1 of sequence i of a pool: [h_kv, n, e]."""
    pool = getattr(st, name).cpu().numpy()
    pages = st.page_table[i].cpu().numpy()[: -(-n // st.page_size)]
    return np.concatenate([pool[p] for p in pages], 1)[:, :n] if n else pool[0][:, :0]


def _check_pools(st, i, K, V, k_exp=0, v_exp=0):
    """Sequence i holds exactly the quantised K, V [n, h, d] (float64)."""
    for x, exp, c, keys in ((K, k_exp, "k", True), (V, v_exp, "v", False)):
        codes, scales = R.quantise(x.transpose(1, 0, 2), exp)
        assert np.array_equal(_gather(st, c + "_scales", i, len(x)), R.e4m3_bytes(scales)), (c, i)
        finite = np.isfinite(scales)
        got = _gather(st, c + "_codes", i, len(x))
        want = R.rows(codes, keys)
        if finite.all():
            assert np.array_equal(got, want), (c, i)


def _check_summary(st, i, K, B):
    """Summaries of complete chunks and the open chunk's state from keys K [n, h, d] (float64)."""
    n = len(K)
    kbar, state, qbar = st.kbar[i].cpu().numpy(), st.state[i].cpu().numpy(), st.qbar.cpu().numpy().astype(np.float64)
    d = K.shape[2]
    for r in range(K.shape[1]):
        for c in range(n // B):
            k = K[c * B:(c + 1) * B, r]
            ref = R.summary(k, qbar[r])[0]
            # weights: the logit is a sum of d products (d 2^-24 of their absolute sum), then sums of B terms
            dz = 2 * d * 2.0 ** -24 * (np.abs(k) @ np.abs(qbar[r])).max() / math.sqrt(d) * 1.5
            tol = (2 * dz + (2 * B + 64) * 2.0 ** -24) * np.abs(k).max()
            assert np.abs(kbar[r, c] - ref).max() <= tol, (i, r, c)
        assert not kbar[r, n // B:].any()
        k = K[n // B * B:, r]
        if len(k) == 0:
            assert state[r, d] == -np.inf and state[r, d + 1] == 0 and not state[r, :d].any()
            continue
        _, m, l, acc = R.summary(k, qbar[r])
        dz = 2 * d * 2.0 ** -24 * (np.abs(k) @ np.abs(qbar[r])).max() / math.sqrt(d) * 1.5
        rel = 2 * dz + (2 * B + 64) * 2.0 ** -24
        assert abs(state[r, d] - m) <= 2 * dz + 2.0 ** -22 * abs(m)
        assert abs(state[r, d + 1] - l) <= 2 * rel * l
        assert np.abs(state[r, :d] - acc).max() <= 2 * rel * l * np.abs(k).max()


@pytest.mark.parametrize("d,hkv,B,page", [(128, 2, 64, 128), (64, 3, 32, 64), (128, 1, 16, 48), (64, 8, 128, 128)])
def test_append_in_pieces(d, hkv, B, page):
    """Pieces of 1 token, of a few, across one and several chunk and page borders, ragged counts with zeros; the
    pools, summaries and states equal the definition's, read-back is exact, other pages stay untouched."""
    rng = np.random.default_rng(d + B)
    b, cap = 3, 6 * page + B
    st = _state(rng, b, cap, 2 * hkv, hkv, d, chunk=B, page=page, k_exp=1, v_exp=-3)
    st.k_codes.fill_(7)
    st.v_scales.fill_(9)
    K, V = _bf16(rng, b, cap, hkv, d), _bf16(rng, b, cap, hkv, d, scale=0.1)
    K[:, :, :, 3] *= 30   # an outlier channel
    K[0, 5, 0, :32] = 0   # an empty group
    held = np.zeros(b, int)
    for n, counts in [(1, [1, 1, 1]), (3, [3, 0, 2]), (4, [4, 4, 4]), (5, [5, 1, 0]), (B, [B, B - 1, 3]), (1, [1, 1, 1]),
                      (2 * B + 7, [2 * B + 7, B, 1]), (6 * page, [page + 1, 2 * page, 0])]:
        counts = np.minimum(counts, cap - held)
        k = torch.zeros(b, n, hkv, d, dtype=torch.bfloat16)
        v = torch.full((b, n, hkv, d), NAN, dtype=torch.bfloat16)   # beyond counts: never read into anything
        for i, c in enumerate(counts):
            k[i, :c], v[i, :c] = K[i, held[i]:held[i] + c], V[i, held[i]:held[i] + c]
        st.append(k.cuda(), v.cuda(), torch.tensor(counts, dtype=torch.int32).cuda())
        held += counts
        assert st.seqlens.tolist() == held.tolist()
    Kd, Vd = K.double().numpy(), V.double().numpy()
    for i in range(b):
        _check_pools(st, i, Kd[i, :held[i]], Vd[i, :held[i]], 1, -3)
        _check_summary(st, i, Kd[i, :held[i]], B)
    # rows behind the last token and pages outside the table are as they were
    used = set(st.page_table.flatten().tolist())
    for p in set(range(st.k_codes.shape[0])) - used:
        assert (st.k_codes[p] == 7).all() and (st.v_scales[p] == 9).all()
    i = int(held.argmin())
    assert (st.k_codes[st.page_table[i, held[i] // page].item(), :, held[i] % page:] == 7).all()
    # read-back: exact values, zeros outside 0..length-1
    start = torch.tensor([-2, 0, int(held[2]) - 3], dtype=torch.int32).cuda()
    n = 2 * B + 11
    K2, V2 = st.load(start, n)
    for i in range(b):
        for x, y, exp in ((Kd, K2, 1), (Vd, V2, -3)):
            codes, s = R.quantise(x[i, :held[i]], exp)
            want = np.zeros((n,) + x.shape[2:])
            at = start[i].item() + np.arange(n)
            ok = (at >= 0) & (at < held[i])
            want[ok] = R.values(codes, s, exp)[at[ok]]
            assert np.array_equal(y[i].double().cpu().numpy(), want), i


def test_one_at_a_time_equals_at_once():
    """Codes, scales and lengths are the same whether tokens come one by one or together."""
    rng = np.random.default_rng(0)
    b, n, hkv, d, B, page = 2, 150, 2, 128, 32, 64
    K, V = _bf16(rng, b, n, hkv, d).cuda(), _bf16(rng, b, n, hkv, d).cuda()
    one, all_ = (_state(np.random.default_rng(1), b, 192, 4, hkv, d, chunk=B, page=page) for _ in range(2))
    for t in range(n):
        one.append(K[:, t], V[:, t])
    all_.append(K, V)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales", "seqlens"):
        assert torch.equal(getattr(one, name), getattr(all_, name)), name
    _check_summary(one, 1, K[1].double().cpu().numpy(), B)
    _check_summary(all_, 1, K[1].double().cpu().numpy(), B)


def test_special_values():
    """Zeros, values below the smallest and above the largest scale, ties, infinities and NaNs."""
    rng = np.random.default_rng(3)
    st = _state(rng, 1, 64, 1, 1, 64, chunk=32, page=64)
    K = torch.zeros(1, 40, 1, 64, dtype=torch.bfloat16)
    K[0, 1] = 1e-5                                     # the scale rounds to 0
    K[0, 2] = 0.0137 * torch.linspace(-1, 1, 64)       # the smallest scale
    K[0, 3] = 3e38                                     # the largest scale, clipped
    K[0, 4, 0, :32] = torch.arange(-16, 16) / 2        # halves: ties of scale 1.125
    K[0, 5, 0, 0] = 7.0                                # scale 1: ties at every half
    K[0, 5, 0, 1:16] = torch.arange(15) - 6.5
    K[0, 6, 0, 40] = NAN
    K[0, 7, 0, 2] = float("inf")
    K[0, 8, 0, 2] = -float("inf")
    K[0, 9] = -0.0
    for t in range(10, 40):
        K[0, t] = _bf16(rng, 1, 64, scale=2.0 ** (t - 25))
    V = K.flip(1).clone()
    st.append(K.cuda(), V.cuda())
    _check_pools_finite(st, K[0].double().numpy(), V[0].double().numpy())
    K2, V2 = st.load(0, 40)
    for x, y in ((K, K2), (V, V2)):
        codes, s = R.quantise(x[0].double().numpy(), 0)
        assert np.array_equal(y[0].double().cpu().numpy(), R.values(codes, s, 0), equal_nan=True)
    assert torch.isnan(K2[0, 6, 0, 32:]).all() and torch.isfinite(K2[0, 6, 0, :32]).all()


def _check_pools_finite(st, K, V):
    for x, c, keys in ((K, "k", True), (V, "v", False)):
        codes, scales = R.quantise(x.transpose(1, 0, 2), 0)
        assert np.array_equal(_gather(st, c + "_scales", 0, len(x)), R.e4m3_bytes(scales))
        ok = np.isfinite(scales).all(-1)
        assert np.array_equal(_gather(st, c + "_codes", 0, len(x))[ok], R.rows(codes, keys)[ok])


def test_append_limits():
    """Counts below 0 and above n, tokens beyond the capacity, unmapped pages, strided inputs."""
    rng = np.random.default_rng(4)
    b, cap, hkv, d, B, page = 4, 100, 2, 64, 32, 32
    st = _state(rng, b, cap, 2, hkv, d, chunk=B, page=page)
    big = _bf16(rng, b, 20, 2, hkv, 2 * d).cuda()
    k, v = big[:, :, 0, :, :d], big[:, :, 1, :, d:]
    st.append(k, v, torch.tensor([-3, 99, 20, 7], dtype=torch.int32).cuda())
    assert st.seqlens.tolist() == [0, 20, 20, 7]
    kd, vd = k.double().cpu().numpy(), v.double().cpu().numpy()
    for i, n in enumerate([0, 20, 20, 7]):
        _check_pools(st, i, kd[i, :n], vd[i, :n])
    more = _bf16(rng, b, 90, hkv, d).cuda()
    st.page_table[3, 2] = -1          # positions 64..95 of sequence 3
    st.page_table[2, 1] = 10 ** 6     # beyond the pool: positions 32..63 of sequence 2
    before = st.k_codes.clone()
    st.append(more, more)
    assert st.seqlens.tolist() == [90, 100, 100, 97]
    m = more.double().cpu().numpy()
    _check_pools(st, 0, m[0], m[0])
    _check_pools(st, 1, np.concatenate([kd[1, :20], m[1, :80]]), np.concatenate([vd[1, :20], m[1, :80]]))
    K2, _ = st.load(0, cap)
    assert not K2[3, 64:96].any() and not K2[2, 32:64].any() and K2[3, 96].any() and K2[2, 64].any()
    free = set(range(st.k_codes.shape[0])) - set(st.page_table.flatten().tolist())
    for p in free:
        assert torch.equal(st.k_codes[p], before[p])
    _check_summary(st, 2, np.concatenate([kd[2, :20], m[2, :80]]), B)   # summaries do not need the pages
    st.append(more, more)
    assert st.seqlens.tolist() == [100] * 4
    st.append(more[:, :0], more[:, :0])
    assert st.seqlens.tolist() == [100] * 4


def _fill_ref(rng, b, lens, hkv, d, k_size=1.0, v_size=1.0):
    n = max(max(lens), 1)
    K, V = _bf16(rng, b, n, hkv, d, scale=k_size), _bf16(rng, b, n, hkv, d, scale=v_size)
    K[..., 7] *= 6
    return K, V


def _decode_ref(st, q, K, V, lens, hq, hkv, d, B, route, k_exp, v_exp):
    """float64 outputs and error bounds from the quantised values and the given routes."""
    g = hq // hkv
    out, err = np.zeros((len(lens), hq, d)), np.zeros((len(lens), hq, d))
    for i, n in enumerate(lens):
        if n == 0:
            continue
        ck, sk = R.quantise(K[i, :n], k_exp)
        cv, sv = R.quantise(V[i, :n], v_exp)
        kk, vv = R.values(ck, sk, k_exp), R.values(cv, sv, v_exp)
        own = (n - 1) // B
        for r in range(hkv):
            bias = np.full(n, -np.inf)
            if route is None:
                bias[:] = 0
            else:
                cnt, idx, bs = (t[i, r] for t in route)
                for e in range(cnt):
                    bias[idx[e] * B:(idx[e] + 1) * B] = bs[e]
            bias[own * B:] = 0
            o, e = R.attend(q[i, r * g:(r + 1) * g], kk[:, r], vv[:, r], bias, sk[:, r] * 2.0 ** k_exp, sv[:, r] * 2.0 ** v_exp)
            out[i, r * g:(r + 1) * g], err[i, r * g:(r + 1) * g] = o, e
    return out, err


def _check_out(o, ref, err):
    o = o.double().cpu().numpy()
    tol = err + 2.0 ** -8 * np.abs(ref) + 2.0 ** -133
    bad = ~(np.abs(o - ref) <= tol)
    assert not bad.any(), (int(bad.sum()), np.abs(o - ref)[bad][:4], tol[bad][:4], np.argwhere(bad)[:4])


CASES = [
    # hq, hkv, d, B, page, lengths
    (8, 1, 128, 64, 128, [1]),
    (2, 2, 128, 64, 64, [15, 16, 17, 64, 65]),
    (4, 2, 64, 32, 64, [1, 31, 32, 33, 500]),
    (8, 2, 64, 16, 48, [0, 47, 48, 49, 0, 300]),
    (32, 4, 128, 128, 256, [129, 1000, 127]),
    (32, 2, 128, 64, 128, [2500, 1]),
    (16, 1, 64, 64, 64, [700, 64, 3]),
    (16, 16, 64, 16, 16, [100, 257]),
    (64, 8, 128, 32, 32, [40, 0, 1111]),
    (16, 1, 128, 16, 64, [333, 16]),
    (4, 1, 128, 16, 32, [17, 200, 0, 15]),
    (16, 1, 64, 16, 16, [100, 1]),
    (16, 4, 64, 128, 128, [128, 129, 1500]),
]


@pytest.mark.parametrize("dense", [True, False])
@pytest.mark.parametrize("hq,hkv,d,B,page,lens", CASES)
def test_decode(hq, hkv, d, B, page, lens, dense):
    rng = np.random.default_rng(len(lens) * 1000 + hq + d)
    b, cap = len(lens), -(-max(lens) // page) * page + B
    st = _state(rng, b, cap, hq, hkv, d, chunk=B, page=page, alpha=1.5, gamma=0.0 if dense else 3.0, k_exp=-1, v_exp=2)
    # what lies behind the last token is not zero
    for t in (st.k_codes, st.k_scales, st.v_codes, st.v_scales):
        t.random_(0, 256)
    st.v_scales.fill_(0x7f)   # NaN
    K, V = _fill_ref(rng, b, lens, hkv, d, v_size=3.0)
    st.fill(K.cuda(), V.cuda(), lens)
    q = _bf16(rng, b, hq, d, scale=1.5)
    route = None
    if not dense:
        counts = torch.zeros(b, hkv, dtype=torch.int32, device="cuda")
        idx = torch.zeros(b, hkv, st.T, dtype=torch.int32, device="cuda")
        bias = torch.zeros(b, hkv, st.T, device="cuda")
        st.route = D.route_out(counts, idx, bias)
    o = st.decode(q.cuda()).clone()
    if not dense:
        route = tuple(t.cpu().numpy() for t in (counts, idx, bias))
        for i, n in enumerate(lens):
            assert all(0 < route[0][i, r] or n <= B for r in range(hkv))
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), lens, hq, hkv, d, B, route, -1, 2)
    _check_out(o, ref, err)
    for i, n in enumerate(lens):
        if n == 0:
            assert not o[i].any()
    st.route = None   # the route output changes nothing, and neither does a second call
    assert torch.equal(st.decode(q.cuda()), o)


def test_decode_long_equals_dequantised():
    """A long dense row over many blocks: against float64 attention over the values read back."""
    rng = np.random.default_rng(11)
    b, n, hq, hkv, d, B, page = 2, 70001, 16, 2, 128, 64, 128
    st = _state(rng, b, n + 63, hq, hkv, d, chunk=B, page=page, gamma=0.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    K = torch.randn(b, n, hkv, d, device="cuda", generator=g).bfloat16()
    V = torch.randn(b, n, hkv, d, device="cuda", generator=g).bfloat16()
    lens = [n, 333]
    st.fill(K, V, lens)
    q = _bf16(rng, b, hq, d, scale=2.0).cuda()
    o = st.decode(q)
    K2, V2 = st.load(0, n)
    for i, m in enumerate(lens):
        for r in range(hkv):
            k, v = K2[i, :m, r].double().cpu().numpy(), V2[i, :m, r].double().cpu().numpy()
            # upper bounds of the scales (max / scale >= 6.5)
            ks, vs = (np.abs(x).reshape(m, -1, 32).max(2) / 6.5 for x in (k, v))
            ref, err = R.attend(q[i, r * 8:(r + 1) * 8].double().cpu().numpy(), k, v, np.zeros(m), ks, vs)
            _check_out(o[i, r * 8:(r + 1) * 8], ref, err)


def test_decode_nonfinite():
    """A NaN or an infinity in an attended key or value reaches the outputs of its KV head only; one behind the
    last token, or in a chunk's place that the table does not map, does not."""
    rng = np.random.default_rng(12)
    b, hq, hkv, d, B, page = 3, 8, 2, 128, 32, 64
    st = _state(rng, b, 256, hq, hkv, d, chunk=B, page=page, gamma=0.0)
    K, V = _bf16(rng, b, 200, hkv, d), _bf16(rng, b, 200, hkv, d)
    V[0, 50, 0, 3] = float("inf")
    K[1, 120, 1, 64] = NAN
    K[2, 199], V[2, 199] = NAN, NAN
    st.fill(K.cuda(), V.cuda(), [200, 200, 200])
    st.seqlens[2] = 199
    o = st.decode(_bf16(rng, b, hq, d).cuda())
    assert torch.isnan(o[0, :4, :32]).all() and torch.isfinite(o[0, :4, 32:]).all() and torch.isfinite(o[0, 4:]).all()
    assert torch.isnan(o[1, 4:]).all() and torch.isfinite(o[1, :4]).all()
    assert torch.isfinite(o[2]).all()


def test_unmapped_pages_count_as_zeros():
    rng = np.random.default_rng(13)
    b, hq, hkv, d, B, page, n = 1, 4, 1, 64, 16, 32, 150
    st = _state(rng, b, 160, hq, hkv, d, chunk=B, page=page, gamma=0.0)
    K, V = _bf16(rng, b, n, hkv, d), _bf16(rng, b, n, hkv, d)
    st.fill(K.cuda(), V.cuda(), [n])
    st.page_table[0, 1] = -1
    st.page_table[0, 3] = st.k_codes.shape[0]
    o = st.decode(_q := _bf16(rng, b, hq, d).cuda())
    K2, V2 = (t[0, :, 0].double().cpu().numpy() for t in st.load(0, n))
    assert not K2[32:64].any() and not V2[96:128].any()
    ks, vs = (np.abs(x).reshape(n, -1, 32).max(2) / 6.5 for x in (K2, V2))
    ref, err = R.attend(_q[0].double().cpu().numpy(), K2, V2, np.zeros(n), ks, vs)
    _check_out(o[0], ref, err)


def test_large_logits_and_moving_maximum():
    """Logits of several hundred, and keys that grow along the sequence, so that the softmax's reference moves often."""
    rng = np.random.default_rng(14)
    hq, hkv, d, B, page, n = 16, 1, 128, 64, 64, 1500
    st = _state(rng, 1, 1536, hq, hkv, d, chunk=B, page=page, gamma=0.0, k_exp=4)
    K, V = _bf16(rng, 1, n, hkv, d), _bf16(rng, 1, n, hkv, d)
    K = (K.double() * torch.linspace(0.01, 40, n)[None, :, None, None]).bfloat16()
    st.fill(K.cuda(), V.cuda(), [n])
    q = _bf16(rng, 1, hq, d, scale=2.0)
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), [n], hq, hkv, d, B, None, 4, 0)
    _check_out(st.decode(q.cuda()), ref, err)


@pytest.mark.parametrize("d,B,hq", [(128, 64, 8), (128, 16, 16), (64, 32, 4), (64, 16, 16)])
def test_value_scales_of_all_sizes(d, B, hq):
    """Values whose scales reach from the smallest to the largest, growing, falling or mixed along the sequence, each
    output to within its bound; and a NaN among small values stays in its group."""
    rng = np.random.default_rng(31)
    n, b = 700, 4
    st = _state(rng, b, 704, hq, 1, d, chunk=B, page=64, gamma=0.0)
    size = np.exp2(np.linspace(-6.5, 11.5, n))
    K, V = _bf16(rng, b, n, 1, d, scale=0.5), _bf16(rng, b, n, 1, d)
    order = [np.arange(n), np.arange(n)[::-1], rng.permutation(n)]
    for i in range(3):
        V[i] = (V[i].float() * torch.from_numpy(size[order[i]]).float().view(n, 1, 1)).bfloat16()
    V[3] = (V[3].float() * 2.0 ** -6).bfloat16()
    st.fill(K.cuda(), V.cuda(), [n] * b)
    q = _bf16(rng, b, hq, d)
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), [n] * b, hq, 1, d, B, None, 0, 0)
    _check_out(st.decode(q.cuda()), ref, err)
    V[3, 100, 0, 40] = NAN
    st.fill(K.cuda(), V.cuda(), [n] * b)
    o = st.decode(q.cuda())
    assert torch.isnan(o[3, :, 32:64]).all()
    rest = [e for e in range(d) if not 32 <= e < 64]
    _check_out(o[3:][..., rest], ref[3:][..., rest], err[3:][..., rest])


def test_small_values_beside_a_strong_key():
    """One key outweighs each of 3000 others by 2^16; their values are small, all of one sign, and still count."""
    rng = np.random.default_rng(32)
    n, hq, d, B = 3001, 4, 128, 64
    st = _state(rng, 1, 3008, hq, 1, d, chunk=B, page=64, gamma=0.0)
    K, V = torch.zeros(1, n, 1, d, dtype=torch.bfloat16), torch.full((1, n, 1, d), 2.0 ** -6, dtype=torch.bfloat16)
    K[0, 5] = 1.0
    V[0, 5] = 0.0
    q = torch.full((1, hq, d), 11.0 / np.sqrt(d), dtype=torch.bfloat16)   # logit 11
    st.fill(K.cuda(), V.cuda(), [n])
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), [n], hq, 1, d, B, None, 0, 0)
    assert err.max() < 0.3 * ref.min()   # the bound would notice if they were lost
    _check_out(st.decode(q.cuda()), ref, err)


@pytest.mark.parametrize("hq,hkv,d,B,lens", [(8, 2, 64, 32, [900, 0, 257, 1]), (16, 1, 128, 16, [400, 33, 0]),
                                             (32, 2, 128, 128, [0, 500, 129]), (16, 4, 128, 64, [700] * 40 + [0, 3])])
@pytest.mark.parametrize("gamma", [0.0, 3.0])
def test_short_and_long_capacity(hq, hkv, d, B, lens, gamma):
    """The same sequences in a cache just long enough (a block per pair) and in a long one (shared list and merge):
    both within their bounds, zeros for the empty ones, and the routes the same."""
    rng = np.random.default_rng(33)
    b, n, page = len(lens), max(lens), 128
    K, V, q = _bf16(rng, b, n, hkv, d), _bf16(rng, b, n, hkv, d), _bf16(rng, b, hq, d)
    qbar = torch.from_numpy(rng.standard_normal((hkv, d)).astype(np.float32) * 0.3).cuda()
    routes = []
    for cap in (n, 9000):
        st = _state(np.random.default_rng(34), b, cap, hq, hkv, d, chunk=B, page=page, gamma=gamma)
        st.qbar = qbar   # (_state draws the table first, which depends on the capacity)
        T = cap // B
        rt = [torch.zeros(b, hkv, dtype=torch.int32, device="cuda"), torch.zeros(b, hkv, T, dtype=torch.int32, device="cuda"),
              torch.zeros(b, hkv, T, device="cuda")]
        if gamma:
            st.route = D.route_out(*rt)
        st.fill(K.cuda(), V.cuda(), lens)
        o = st.decode(q.cuda())
        route = [t.cpu().numpy() for t in rt] if gamma else None
        ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), lens, hq, hkv, d, B, route, 0, 0)
        _check_out(o, ref, err)
        assert all(not o[i].any() for i, m in enumerate(lens) if m == 0)
        if gamma:
            routes.append([set(route[1][i, r, :route[0][i, r]]) for i in range(b) for r in range(hkv)])
    if gamma:   # the two ways of routing round differently: a chunk at the threshold may change sides
        assert sum(x != y for x, y in zip(*routes)) <= max(1, len(routes[0]) // 20)


def test_steps_graph_and_streams():
    """append + decode replayed from a graph over page and chunk borders equals eager steps; a call on another stream
    gives the same; two captured graphs of two caches do not disturb each other."""
    rng = np.random.default_rng(15)
    b, hq, hkv, d, B, page = 3, 16, 2, 128, 64, 64
    make = lambda: _state(np.random.default_rng(16), b, 512, hq, hkv, d, chunk=B, page=page, gamma=3.0)   # noqa: E731
    eager, graph, other = make(), make(), make()
    K, V = _bf16(rng, b, 300, hkv, d).cuda(), _bf16(rng, b, 300, hkv, d).cuda()
    Q = _bf16(rng, 300, b, hq, d).cuda()
    lens = [130, 60, 0]
    for st in (eager, graph, other):
        st.fill(K[:, :130], V[:, :130], lens)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for t in range(130, 270):
        a = eager.step(Q[t], K[:, t], V[:, t]).clone()
        g = graph.graph_step(Q[t], K[:, t], V[:, t]).clone()
        stream.wait_stream(torch.cuda.current_stream())
        o = other.step(Q[t], K[:, t], V[:, t], stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
        assert torch.equal(a, g) and torch.equal(a, o), t
    for name in ("k_codes", "v_codes", "k_scales", "v_scales", "kbar", "state", "seqlens"):
        assert torch.equal(getattr(eager, name), getattr(graph, name)), name
        assert torch.equal(getattr(eager, name), getattr(other, name)), name


@pytest.mark.parametrize("cap", [256, 9984])
def test_length_beyond_the_capacity(cap):
    """A length that someone set too large counts as the capacity: no chunk is attended twice."""
    rng = np.random.default_rng(35)
    K, V, q = _bf16(rng, 2, cap, 2, 64), _bf16(rng, 2, cap, 2, 64), _bf16(rng, 2, 4, 64)
    st = _state(rng, 2, cap, 4, 2, 64, chunk=32, page=64, gamma=2.0)
    st.fill(K.cuda(), V.cuda(), [cap, cap])
    o = st.decode(q.cuda()).clone()
    st.seqlens += torch.tensor([1, 10 ** 6], dtype=torch.int32, device="cuda")
    assert torch.equal(st.decode(q.cuda()), o)


def test_graph_refuses_other_shapes():
    """A recorded step takes the sizes and type it was recorded with: nothing is broadcast or converted."""
    rng = np.random.default_rng(28)
    st = _state(rng, 2, 128, 4, 2, 64, chunk=32, page=32)
    q, k = _bf16(rng, 2, 4, 64).cuda(), _bf16(rng, 2, 2, 64).cuda()
    st.graph_step(q, k, k)
    before = st.graph_step(q, k, k).clone()
    for bad in ((q[:1], k, k), (q, k[:1], k), (q, k, k.float()), (q, k, k[:, :, :1])):
        with pytest.raises(ValueError):
            st.graph_step(*bad)
    assert st.seqlens.tolist() == [2, 2] and torch.equal(st.O, before)


def test_cache_shorter_than_a_chunk():
    """No chunk ever completes: no summaries, and routed attention is attention over the own chunk."""
    rng = np.random.default_rng(29)
    cap, n, hq, hkv, d = 20, 17, 4, 2, 64
    K, V, q = _bf16(rng, 2, n, hkv, d), _bf16(rng, 2, n, hkv, d), _bf16(rng, 2, hq, d)
    out = []
    for gamma in (3.0, 0.0):
        st = _state(np.random.default_rng(30), 2, cap, hq, hkv, d, chunk=32, page=32, gamma=gamma)
        st.fill(K[:, :n - 1].cuda(), V[:, :n - 1].cuda(), [n - 1, 0])
        counts = torch.full((2, hkv), 7, dtype=torch.int32, device="cuda")
        st.route = D.route_out(counts)
        st.append(K[:, n - 1].cuda(), V[:, n - 1].cuda())
        out.append(st.decode(q.cuda()).clone())
        assert not counts.any() and st.seqlens.tolist() == [n, 1]
        for i, m in enumerate((n, 1)):
            _check_pools(st, i, K[i, n - m:].double().numpy(), V[i, n - m:].double().numpy())
    ref, err = _decode_ref(st, q.double().numpy(), np.stack([K[0].double().numpy(), np.roll(K[1].double().numpy(), 1, 0)]),
                           np.stack([V[0].double().numpy(), np.roll(V[1].double().numpy(), 1, 0)]), [n, 1], hq, hkv, d, 32,
                           None, 0, 0)
    _check_out(out[0], ref, err)
    assert torch.equal(*out)


def test_matches_bf16_cache_routes():
    """The 4-bit cache routes as the bf16 paged cache does (same summaries), step after step, and its outputs stay
    within the quantisation's distance."""
    rng = np.random.default_rng(17)
    b, hq, hkv, d, B, page, cap = 2, 16, 2, 128, 64, 128, 1024
    st = _state(rng, b, cap, hq, hkv, d, chunk=B, page=page, gamma=3.0)
    ref = D.PagedDecodeState(b, cap, hq, hkv, d, chunk=B, alpha=1.5, gamma=3.0, page_size=page,
                             num_pages=st.k_codes.shape[0], page_table=st.page_table, qbar=st.qbar)
    K, V = _bf16(rng, b, 700, hkv, d).cuda(), _bf16(rng, b, 700, hkv, d).cuda()
    st.fill(K[:, :600], V[:, :600], [600, 555])
    ref.fill(K[:, :600], V[:, :600], [600, 555])
    outs = []
    for s in (st, ref):
        rt = [torch.zeros(b, hkv, dtype=torch.int32, device="cuda"),
              torch.full((b, hkv, cap // B), -1, dtype=torch.int32, device="cuda"),
              torch.zeros(b, hkv, cap // B, device="cuda")]
        s.route = D.route_out(*rt)
        s.rt = rt
    for t in range(600, 640):
        q = _bf16(rng, b, hq, d).cuda()
        o = [s.step(q, K[:, t].contiguous(), V[:, t].contiguous()).double() for s in (st, ref)]
        outs.append(o)
        assert torch.equal(st.rt[0], ref.rt[0]) and torch.equal(st.rt[1], ref.rt[1])
    # 4 bits with groups of 32: about a tenth of the values' size per key and value, averaged down
    far = sum((a - c).norm() for a, c in outs) / sum(c.norm() for _, c in outs)
    assert far < 0.25, far


def test_decode_more_pairs_than_blocks():
    """More (sequence, KV head) pairs than the GPU has room for blocks, some of them empty."""
    rng = np.random.default_rng(20)
    b, hq, hkv, d, B, page = 130, 16, 4, 64, 32, 64
    lens = [int(n) for n in rng.integers(0, 140, b)]
    lens[5], lens[6] = 0, 1
    st = _state(rng, b, 192, hq, hkv, d, chunk=B, page=page, gamma=0.0)
    K, V = _fill_ref(rng, b, lens, hkv, d)
    st.fill(K.cuda(), V.cuda(), lens)
    q = _bf16(rng, b, hq, d)
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), lens, hq, hkv, d, B, None, 0, 0)
    _check_out(st.decode(q.cuda()), ref, err)
    st.seqlens.zero_()
    assert not st.decode(q.cuda()).any()      # nothing cached at all


@pytest.mark.parametrize("size", [1e-37, 1e-3, 1e3, 1e30])
def test_query_sizes(size):
    """Queries of any size: with keys to match, the softmax is the same."""
    rng = np.random.default_rng(21)
    hq, hkv, d, B, page, n = 8, 1, 128, 64, 64, 300
    st = _state(rng, 1, 320, hq, hkv, d, chunk=B, page=page, gamma=0.0)
    K, V = _bf16(rng, 1, n, hkv, d), _bf16(rng, 1, n, hkv, d)
    st.fill(K.cuda(), V.cuda(), [n])
    q = _bf16(rng, 1, hq, d, scale=size)
    q[0, 1], q[0, 2, 5:] = 0, 0           # a head without a query: the mean of the values; one of few elements
    q[0, 3, 7] = size * 1e-6              # elements of very different size
    if size > 1e29:
        q[0, 0] = 0
        q[0, 0, 0] = 3e38                 # logits beyond fp32
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), [n], hq, hkv, d, B, None, 0, 0)
    o = st.decode(q.cuda())
    _check_out(o[:, 1:2], ref[:, 1:2], err[:, 1:2])
    if size < 1e29:
        _check_out(o, ref, err)


def test_nonfinite_queries_stay_in_their_heads():
    rng = np.random.default_rng(22)
    hq, hkv, d, B, page, n = 16, 1, 64, 32, 32, 100
    st = _state(rng, 2, 128, hq, hkv, d, chunk=B, page=page, gamma=0.0)
    K, V = _bf16(rng, 2, n, hkv, d), _bf16(rng, 2, n, hkv, d)
    st.fill(K.cuda(), V.cuda(), [n, n])
    q = _bf16(rng, 2, hq, d).cuda()
    clean = st.decode(q).clone()
    q[0, 3, 10], q[1, 9, 0] = NAN, float("inf")
    o = st.decode(q)
    assert torch.isnan(o[0, 3]).all() and torch.isnan(o[1, 9]).all()
    keep = torch.ones(2, hq, dtype=torch.bool)
    keep[0, 3] = keep[1, 9] = False
    assert torch.equal(o[keep], clean[keep])


def test_far_pages():
    """A pool whose pages lie more than 2^31 bytes apart, and page strides larger than a page."""
    rng = np.random.default_rng(23)
    hq, hkv, d, B, page, n = 4, 2, 128, 64, 64, 200
    st = _state(rng, 1, 256, hq, hkv, d, chunk=B, page=page, gamma=0.0, slack=0)
    near = _state(np.random.default_rng(23), 1, 256, hq, hkv, d, chunk=B, page=page, gamma=0.0, slack=0)
    size = hkv * page * d // 2
    stride = (1 << 30) + 4096
    far = torch.zeros(3 * stride + size, dtype=torch.uint8, device="cuda")
    st.k_codes = torch.as_strided(far, (4, hkv, page, d // 2), (stride, page * d // 2, d // 2, 1))
    st.kv = D.q4_kv(st.k_codes, st.k_scales, st.v_codes, st.v_scales, st.page_table, page_size=page)
    st.qbar = near.qbar
    K, V = _bf16(rng, 1, n, hkv, d).cuda(), _bf16(rng, 1, n, hkv, d).cuda()
    q = _bf16(rng, 1, hq, d).cuda()
    outs = []
    for s in (st, near):
        s.fill(K, V, [n])
        outs.append((s.decode(q).clone(), *s.load(0, n)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)
    pool = D.PagePool.of([near])
    far_pool = D.PagePool.of([st])
    for s, p in ((near, pool), (st, far_pool)):
        p.refs.zero_()
        p.copy([s.page_table[0, 0].item()], [s.page_table[0, 1].item()])
    assert torch.equal(st.load(0, n)[0], near.load(0, n)[0])


def test_refusals():
    rng = np.random.default_rng(24)
    st = _state(rng, 2, 128, 4, 2, 64, chunk=32, page=32)
    k = _bf16(rng, 2, 3, 2, 64).cuda()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
    for bad in (lambda: st.append(k.float(), k), lambda: st.append(k.cpu(), k), lambda: st.append(k, k, ints(1, 2).long()),
                lambda: st.append(k, None), lambda: st.decode(k), lambda: st.decode(st.O.float()), lambda: st.load(ints(0, 0).cpu(), 3),
                lambda: st.append(k[0, 0], k[0, 0])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: st.append(k, k[:, :2]), lambda: st.append(k[:1], k[:1]), lambda: st.append(k, k, ints(1)),
                lambda: st.append(k.transpose(2, 3), k.transpose(2, 3)), lambda: st.append(k, k, ints(1, 0, 2, 0)[::2]), lambda: st.load(1 << 32, 3), lambda: st.load(-(1 << 31) - 1, 3),
                lambda: st.load(ints(0), 3), lambda: st.load(0, 3, k[:, :2], k), lambda: st.decode(torch.zeros_like(st.O).transpose(0, 1))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(D.DashError):
        st.load(0, 3, k[:, :1].expand(-1, 3, -1, -1), k)      # all tokens in one place
    with pytest.raises(D.DashError):
        st.append(torch.zeros(2, 3, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64], k)   # rows 136 bytes apart
    for bad in (st.qbar.double(), st.qbar.cpu(), st.qbar.T.contiguous().T, st.qbar[:1]):
        with pytest.raises((TypeError, ValueError)):
            st.qbar = bad
    st.qbar = None
    with pytest.raises(TypeError):
        st.append(k, k)
    st.load(0, 3, None, torch.empty(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        st.load(0, 3, None, torch.empty(2, 4, 2, 64, dtype=torch.bfloat16, device="cuda"))
    big = D.Q4DecodeState(2, 64, 2, 1, 64, chunk=32, alpha=3.0, gamma=1.0, page_size=32)
    with pytest.raises(D.DashError):
        big.decode(big.O.clone())


def test_dense_needs_no_room_for_routing():
    """16 heads x 32768 chunks are more than the routing takes; dense decoding has none."""
    rng = np.random.default_rng(25)
    hq, hkv, d, B, page, n = 16, 1, 64, 16, 64, 500
    kw = dict(chunk=B, page=page)
    st = _state(rng, 1, 524288, hq, hkv, d, gamma=0.0, **kw)
    K, V = _bf16(rng, 1, n, hkv, d), _bf16(rng, 1, n, hkv, d)
    st.fill(K.cuda(), V.cuda(), [n])
    q = _bf16(rng, 1, hq, d)
    ref, err = _decode_ref(st, q.double().numpy(), K.double().numpy(), V.double().numpy(), [n], hq, hkv, d, B, None, 0, 0)
    _check_out(st.decode(q.cuda()), ref, err)
    st = _state(rng, 1, 524288, hq, hkv, d, gamma=1.0, **kw)
    with pytest.raises(D.DashError):
        st.decode(q.cuda())


def test_load_and_append_nothing():
    st = _state(np.random.default_rng(26), 2, 64, 2, 1, 64, chunk=32, page=32)
    K, V = st.load(0, 0)
    assert K.shape == V.shape == (2, 0, 1, 64)
    k = torch.ones(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda")
    st.append(k, k, torch.zeros(2, dtype=torch.int32, device="cuda"))
    st.fill(k, k, [0, 0])
    assert not st.seqlens.any() and not st.k_scales.any() and (st.state[..., 64] == -torch.inf).all()
    assert not st.load(0, 64)[0].any()


@pytest.mark.parametrize("g,hkv,d,B,cap,lens,alpha,gamma,inv_sigma", [
    (8, 2, 128, 64, 2048, [2000, 65, 64], 1.5, 6.0, 1.0),          # 4 warps per head
    (4, 2, 128, 32, 8192, [8000, 1], 2.0, 4.0, 0.5),
    (2, 1, 64, 16, 4096, [4095, 17, 4081], 1.25, 3.0, 1.0),
    (1, 2, 64, 16, 16384, [16000, 9000], 1.5, 8.0, 0.0),           # 2 warps per head
    (16, 1, 128, 16, 32768, [32768, 20000], 1.5, 5.0, 1.0),
    (16, 1, 64, 16, 57600, [57000, 40], 2.0, 5.0, 1.0),            # 8 warps per head
    (8, 1, 64, 16, 40000, [39990], 1.8, 2.0, 1.0),
    (2, 1, 64, 16, 160000, [160000], 1.5, 8.0, 1.0),               # 32 entries per thread
    (1, 1, 64, 16, 320000, [310000], 1.5, 8.0, 1.0),               # more than a block's registers hold
    # one block per row: up to 128, 256 and 512 chunks, the last places and the first beyond
    (4, 2, 64, 32, 1000, [999, 33, 32, 1], 1.5, 3.0, 1.0),
    (16, 1, 128, 16, 2048, [2048, 2033, 16], 1.25, 4.0, 0.5),
    (1, 3, 128, 128, 32767, [32767, 16640], 2.0, 5.0, 1.0),
    (2, 2, 128, 64, 20480, [20480, 20417, 1], 1.5, 6.0, 1.0),
    (8, 1, 128, 64, 20544, [20544], 1.5, 6.0, 1.0),
    (16, 2, 64, 16, 8192, [8192, 4100], 1.5, 6.0, 1.0),
    (8, 2, 64, 16, 8208, [8208, 8191], 2.0, 6.0, 1.0),
])
def test_routes_against_the_oracle(g, hkv, d, B, cap, lens, alpha, gamma, inv_sigma):
    """Routed sets by the margin rule, biases within what the logits' error does to log w, bitmask, for every way the
    routing splits its work."""
    b, T = len(lens), cap // B
    x = inputs.planted(77, b, cap, g * hkv, hkv, d, B, dtype="bf16", chunk_frac=0.05)
    st = D.Q4DecodeState(b, cap, g * hkv, hkv, d, chunk=B, alpha=alpha, gamma=gamma, inv_sigma=inv_sigma, page_size=B * 4,
                         qbar=torch.from_numpy(x["qbar"]).cuda())
    rt = [torch.zeros(b, hkv, dtype=torch.int32, device="cuda"), torch.full((b, hkv, T), -1, dtype=torch.int32, device="cuda"),
          torch.full((b, hkv, T), NAN, device="cuda"), torch.full((b, hkv, (T + 31) // 32), -1, dtype=torch.int32, device="cuda")]
    st.route = D.route_out(*rt)
    n = max(lens)
    st.fill(*(torch.from_numpy(x[k][:, :n]).to("cuda", torch.bfloat16) for k in "KV"), lens)
    q = x["Q"][np.arange(b), np.asarray(lens) - 1]
    st.decode(torch.from_numpy(q).to("cuda", torch.bfloat16))
    counts, idx, bias, mask = (t.cpu().numpy() for t in rt)
    _, ref = oracle.decode(q, x["K"], x["V"], x["qbar"], lens, chunk=B, alpha=alpha, gamma=gamma, inv_sigma=inv_sigma,
                           want_route=True)
    pos = (np.asarray(lens) - 1).reshape(b, 1)
    sets = {(i, r, 0): idx[i, r, :counts[i, r]] for i in range(b) for r in range(hkv)}
    mism, _ = check_routes(sets, ref, B, pos, T)
    for (i, r, _), got in sets.items():
        bits = ((mask[i, r].view(np.uint32)[:, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1)
        assert np.array_equal(np.flatnonzero(bits), got)
        if (i, r, 0) in mism or not len(got):
            continue
        w, margin = ref["w"][i, r, 0, got], ref["margin"][i, r, 0, got]
        want = (np.log(w) - np.log(w).mean()) * inv_sigma
        assert (np.abs(bias[i, r, :len(got)] - want) <= bias_tolerance(margin, alpha, gamma, inv_sigma)).all(), (i, r)
    assert len(mism) <= 1
