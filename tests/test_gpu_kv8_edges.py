"""The 8-bit K/V cache at the ends of its ranges: V scales far apart and at bf16's end, queries
that are not finite, scores of any size, padded rows, rows refused on the device. Bounds as in
test_gpu_kv8."""
import numpy as np
import pytest
import torch

import flow_matching_vla_euler_b200 as V

from .test_gpu_kv8 import Pair, _filled, bf16, host, i32, kv_values

pytestmark = pytest.mark.gpu

# (rows of the call, queries, heads on one K/V head): few and many query rows, items in one part and in several
CALLS = [(1, 1, 1), (1, 10, 2), (1, 40, 2), (160, 10, 2), (160, 40, 2), (100, 80, 2)]


# ---- V scales

SPREADS = [(1e23, 0, 1e23, 0, 0), (1e30, 1e-20, 1, 0, 1e30), (0, 1, 1e25, 1e-17, 1e-5), (1e-20, 1e30, 0, 0, 1e20)]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,nq,H", CALLS)
@pytest.mark.parametrize("spread", range(len(SPREADS)))
def test_v_scales_far_apart(D, B, nq, H, spread):
    """Scores of like size in blocks whose V scales lie up to 2^160 apart, in both orders: each
    key counts in the sum of the weights by its score, whatever its V."""
    rng = np.random.default_rng(spread)
    f = np.repeat(SPREADS[spread], 64)[:, None]
    p = Pair(1, 1, D, 320, 2)
    K, Vv = (rng.standard_normal((1, 2, 320, D)) for _ in range(2))
    p.write(K, Vv * np.stack([f, f[::-1]]))
    slots, lens = rng.integers(0, 2, B), rng.integers(280, 321, B)
    Q = 0.5 * rng.standard_normal((B, nq, H, D))
    p.check_attend(Q, lens, slots=slots)
    Q[:, ::3] *= 1e-6                                # equal scores
    p.check_attend(Q, lens, slots=slots, causal=True, window=200)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,nq,H", CALLS)
def test_v_at_the_end_of_bf16(D, B, nq, H):
    """Averages of values of 2^127 and more, which no partial sum may pass; with scores that
    climb from block to block, so that references lag behind."""
    rng = np.random.default_rng(nq)
    p = Pair(1, 1, D, 320, 2)
    Vv = 2.5e38 * rng.choice([1.0, 0.9, 0.5], (1, 2, 320, D))
    K = rng.standard_normal((1, 2, 320, D))
    p.write(K, Vv)
    Q = 0.5 * rng.standard_normal((B, nq, H, D))
    slots, lens = rng.integers(0, 2, B), rng.integers(280, 321, B)
    p.check_attend(Q, lens, slots=slots)
    f = np.repeat([1.0, 6.0, 12.0, 20.0, 30.0], 64)[:, None]
    p.write(K * f, Vv)
    p.check_attend(Q, lens, slots=slots)
    p.write(np.abs(K) * f, Vv)
    p.check_attend(np.abs(Q), lens, slots=slots, causal=True)


# ---- queries that are not finite

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq", [1, 3, 40])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_infinite_queries_on_keys_of_one_sign(D, nq, bad):
    """All scores of such a row may be -infinity: NaN all the same, unless it sees no key."""
    rng = np.random.default_rng(nq)
    p = Pair(1, 1, D, 200, 1)
    p.write(0.5 + np.abs(rng.standard_normal((1, 1, 200, D))), rng.standard_normal((1, 1, 200, D)))
    Q = rng.standard_normal((4, nq, 4, D))
    Q[0, 0, 1, 3], Q[1, nq - 1, 0], Q[2, 0, 2, D - 1], Q[3, 0, 0, 0] = bad, bad, bad, bad
    lens = [200, 64, 1, 0]
    _, got, ls = p.attend(Q, lens, slots=[0] * 4)
    nan = np.zeros(Q.shape[:3], bool)
    nan[0, 0, 1] = nan[1, nq - 1, 0] = nan[2, 0, 2] = True
    assert np.isnan(got[nan]).all() and np.isnan(ls[nan]).all()
    assert not got[3].any() and np.isneginf(ls[3]).all()
    Q[~np.isfinite(Q)] = 0.0
    _, clean, lc = p.attend(Q, lens, slots=[0] * 4)
    assert np.array_equal(got[~nan], clean[~nan]) and np.array_equal(ls[~nan], lc[~nan])


# ---- rows

@pytest.mark.parametrize("n", [1, 8, 9, 70])
def test_rows_of_no_tokens_are_padding(n):
    """Rows of count 0 name no slot and no position that counts, in writes, reads and attention."""
    rng = np.random.default_rng(n)
    p = _filled(rng, 2, 64, 200, 3, L=2)
    K, Vv = (kv_values(rng, (2, 6, n, 128)) for _ in range(2))
    slots, pos, cnt = [0, 2, 0, 0, -1, 9], [5, 3, 300, 61, 0, -7], [0, n, 0, n, 0, 0]
    p.c.write(bf16(K)[0], bf16(Vv)[0], slots=i32(slots), pos=i32(pos), count=i32(cnt))
    p.c.status()
    p.m.write(bf16(K)[1][:, [1, 3]], bf16(Vv)[1][:, [1, 3]], slots=[2, 0], pos=[3, 61])
    p.check_read(61 + n, slots=[0])
    p.check_read(3 + n, slots=[2])
    out = [torch.full((2, 6, n, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p.c.read(n, slots=i32(slots), pos=i32(pos), count=i32(cnt), K_out=out[0], V_out=out[1])
    p.c.status()
    for w in range(2):
        ref = p.m.read(w, n, slots=[2, 0], pos=[3, 61], batch=2)
        assert np.array_equal(host(out[w])[:, [1, 3]], ref)
        assert torch.all(out[w][:, [0, 2, 4, 5]] == 7.0)
    # nothing to write anywhere
    p.c.write(bf16(K)[0], bf16(Vv)[0], slots=i32([-1] * 6), count=i32([0] * 6))
    p.c.status()


@pytest.mark.parametrize("nq", [1, 4, 60])
def test_rows_of_no_queries_are_padding(nq):
    rng = np.random.default_rng(nq)
    p = _filled(rng, 1, 64, 100, 3)
    Q = rng.standard_normal((5, nq, 2, 64))
    q, out = bf16(Q)[0], torch.full((5, nq, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((5, nq, 2), 9.0, device="cuda")
    p.c.attend(q, i32([-3, 100, 1000, 7, 0]), slots=i32([-1, 2, 5, 0, 0]), q_pos=i32([0, 0, 5000, 0, -9999]),
               q_count=i32([0, nq, 0, nq, 0]), out=out, lse=lse)
    p.c.status()
    assert torch.all(out[[0, 2, 4]] == 7.0) and torch.all(lse[[0, 2, 4]] == 9.0)
    only = p.c.attend(q[[1, 3]], i32([100, 7]), slots=i32([2, 0]), q_pos=i32([0, 0]))
    assert torch.allclose(out[[1, 3]].float(), only.float(), rtol=2.0 ** -6, atol=1e-6)
    # (a count that is out of range is still refused)
    p.c.attend(q, i32([1] * 5), slots=i32([0] * 5), q_count=i32([0, -1, 0, 0, 0]), out=out)
    with pytest.raises(V.VlaError):
        p.c.status()


@pytest.mark.parametrize("nq", [1, 40])
def test_refused_rows_of_a_fresh_tensor_are_zeros(nq):
    rng = np.random.default_rng(nq)
    p = _filled(rng, 1, 64, 100, 3)
    q, _ = bf16(rng.standard_normal((3, nq, 2, 64)))

    def used_memory(shape):                          # what a new tensor may be given next
        old = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        del old

    for kw in (dict(slots=i32([0, 3, 1])), dict(q_pos=i32([0, 101, 0])), dict(kv_len=i32([100, 101, 5]))):
        used_memory(q.shape)
        out = p.c.attend(q, **dict(dict(kv_len=i32([100, 50, 5])), **kw))
        with pytest.raises(V.VlaError):
            p.c.status()
        assert not out[1].any() and out[0].any() and out[2].any()
    for kw in (dict(slots=i32([0, -1, 1])), dict(pos=i32([0, 91, 0]))):
        used_memory((1, 3, 10, 64))
        K, Vv = p.c.read(10, **kw)
        with pytest.raises(V.VlaError):
            p.c.status()
        assert not K[:, 1].any() and not Vv[:, 1].any() and K[:, 0].any() and Vv[:, 2].any()


# ---- refusals

def test_scales_out_of_range_are_refused():
    p = _filled(np.random.default_rng(1), 1, 64, 100, 1)
    q, _ = bf16(np.ones((1, 1, 2, 64)))
    with pytest.raises(ValueError, match="scale"):
        p.c.attend(q, i32([100]), scale=1e-50)       # 0 in fp32, which would stand for the default
    with pytest.raises(V.VlaError) as ei:
        p.c.attend(q, i32([100]), scale=3e38)        # times log2(e): infinite
    assert ei.value.code == V.VLA_ERR_ARG
    p.check_attend(np.ones((1, 1, 2, 64)), [100], scale=1e-40)


def test_more_query_rows_than_an_int_holds_are_refused():
    """2^20 queries of 2048 heads on one K/V head: refused on the host, nothing is launched."""
    p = _filled(np.random.default_rng(2), 1, 64, 64, 1)
    n, out = i32([64]), torch.full((64,), 7.0, dtype=torch.bfloat16, device="cuda")
    a = V.vla_kv8_query()
    a.kv_len, a.batch, a.n_q, a.n_heads = n.data_ptr(), 1, 1 << 20, 2048
    a.q_stride[:], a.out_stride[:] = (0, 0, 8), (8, 8, 8)
    with pytest.raises(V.VlaError, match="query rows") as ei:
        V.vla_kv8_attend(p.c.handle, out.data_ptr(), out.data_ptr(), None, a, torch.cuda.current_stream().cuda_stream)
    assert ei.value.code == V.VLA_ERR_SHAPE
    p.c.status()
    assert torch.all(out == 7.0)


# ---- scores

@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("B,nq,H", [(1, 1, 4), (1, 10, 2), (1, 40, 2), (160, 40, 2), (20, 80, 2)])
def test_scores_of_any_size(D, B, nq, H):
    """Scores from 2^18 to 2^110, of either sign. Each is one product (exact) times the scale, equal
    keys have equal scores and unlike ones differ by 2^-4 of themselves or more, so the softmax is the
    mean over the keys that share the largest. Off by the output's and the weights' rounding to
    bf16, half a step each; lse by two roundings of fp32 and that of the scale, relative."""
    rng = np.random.default_rng(D + nq)
    n = 330
    p = Pair(1, 1, D, n, 2)
    K = np.zeros((1, 2, n, D))
    K[..., 3] = rng.choice([1.0, 1.5, 2.0, 3.5, 7.0], (1, 2, n)) * np.array([1.0, -1.0])[None, :, None]
    p.write(K, rng.standard_normal((1, 2, n, D)))
    Q = np.zeros((B, nq, H, D))
    Q[..., 3] = np.exp2(rng.integers(20, 110, (B, nq, H))) * rng.choice([1.0, -1.0], (B, nq, H))
    slots, lens = rng.integers(0, 2, B), rng.integers(250, n + 1, B)
    for kw in (dict(), dict(causal=True, window=90)):
        _, got, ls = p.attend(Q, lens, slots=slots, **kw)
        ref, rls, mean_v, _, _ = p.m.attend(Q, lens, slots=slots, **kw)
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * mean_v * (1 + 2.0 ** -7))
        assert np.all(np.abs(ls - rls) <= 2.0 ** -21 * np.abs(rls))


@pytest.mark.parametrize("D", [32, 64, 128, 256])
@pytest.mark.parametrize("B,nq,H", CALLS)
def test_a_row_of_one_key_is_that_key(D, B, nq, H):
    """The only weight is 1 whatever its score, so the output is V as it is stored, bit for bit; and
    lse is the score, to the error of the scores (2 e_s for the product's and exp2's)."""
    rng = np.random.default_rng(D + B)
    p = Pair(1, 1, D, 130, 2)
    p.write(kv_values(rng, (1, 2, 130, D)), kv_values(rng, (1, 2, 130, D)))
    slots = rng.integers(0, 2, B)
    Q = 1.5 * rng.standard_normal((B, nq, H, D))
    for lens, kw in ((np.ones(B, int), dict()), (rng.integers(nq, 131, B), dict(causal=True, window=1))):
        qn, got, ls = p.attend(Q, lens, slots=slots, **kw)
        ref, rls, _, mag, _ = p.m.attend(qn, lens, slots=slots, **kw)
        assert np.array_equal(got, ref)
        es = ((D + 8) * 2.0 ** -23 * mag[0] + 2.0 ** -17 * mag[1]) / np.sqrt(D) + 2.0 ** -20
        ok = np.isfinite(rls)
        assert np.array_equal(np.isneginf(ls), ~ok) and np.all(np.abs(ls - rls)[ok] <= 2 * es[ok])
