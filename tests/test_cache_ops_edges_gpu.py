"""Edges of the whole-cache operators that the main tests do not reach:
non-finite values under a vanishing probability, the largest arguments,
selections that mislead the eviction's sample, keys beyond its cache.
"""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO
from test_cache_ops_gpu import Case, _bits, _evict_case, _run_evict

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def abi():
    from block_sparse_attention_kv_b200 import build
    build.build()
    from block_sparse_attention_kv_b200 import abi as m
    return m


def _at(c, s, t):
    return int(c.table[s, t // 16]), t % 16


def _point_at(c, s, t):
    """Token t of sequence s takes every query's attention: its score lies
    above any other by more than 500 (log2 units), so that whatever other
    part of the cache a query meets joins with a factor that is 0 in fp32."""
    q = c.q[s].float().view(c.Hkv, c.Hq // c.Hkv, 128)
    page, slot = _at(c, s, t)
    c.k[page, :, slot] = 150 * (q / q.norm(dim=-1, keepdim=True)).sum(1).bfloat16()


@pytest.mark.parametrize("Hq", [8, 24])
@pytest.mark.parametrize("wide", [False, True])
def test_non_finite_values_under_a_vanishing_probability(abi, Hq, wide):
    """An infinite or NaN value of an attended token makes its channel
    non-finite wherever the sequence is cut, however small its probability."""
    c = Case(abi, [3000, 70], Hq, 2, seed=61, gain=8.0, wide=wide)
    _point_at(c, 0, 1234)
    good = c.want()[0]
    for t, ch, x in ((5, 3, np.inf), (1230, 11, -np.inf), (2100, 40, np.nan), (2999, 77, np.inf)):
        page, slot = _at(c, 0, t)
        c.v[page, :, slot, ch] = x
    c.run()
    c.check()
    got = c.out.float().cpu().numpy()
    odd = np.zeros(128, bool)
    odd[[3, 11, 40, 77]] = True
    assert not np.isfinite(got[0][:, odd]).any()
    assert np.isfinite(got[0][:, ~odd]).all() and np.isfinite(got[1]).all()
    assert np.abs(got[0][:, ~odd] - good[0][:, ~odd]).max() < 0.02


@pytest.mark.parametrize("peak,odd_at", [(700, 100), (100, 700), (700, 639)])
@pytest.mark.parametrize("wide", [False, True])
def test_non_finite_values_across_the_end_of_a_prefix(abi, peak, odd_at, wide):
    c = Case(abi, [900 + i for i in range(5)], 8, 2, shared=640, seed=62, gain=8.0, wide=wide)
    for s in range(5 if peak >= 640 else 1):
        _point_at(c, s, peak)
    page, slot = _at(c, 0, odd_at)
    c.v[page, :, slot, 9] = np.inf
    c.run()
    c.check()
    got = c.out.float().cpu().numpy()
    assert not np.isfinite(got[0, :, 9]).any()
    assert np.isfinite(np.delete(got[0], 9, axis=1)).all()


@pytest.mark.parametrize("pages", [20, 1100])
def test_evict_with_the_largest_keep(abi, pages):
    """keep_tokens 2^31 - 1: every token stays; pages: a block per unit, a cluster per unit."""
    keep = 2 ** 31 - 1
    c = Case(abi, [300], 1, 1, seed=63, max_pages=pages)
    w = torch.rand((1, 1, c.cap), device="cuda")
    w_out = torch.full_like(w, -3.0)
    # a guard of one number behind the list (its length is odd)
    kept = torch.full((keep + 1,), 5, dtype=torch.int32, device="cuda")
    new = torch.zeros_like(c.d_lens)
    k, v = c.k.clone(), c.v.clone()
    ws = abi.alloc_workspace(abi.absp_evict_workspace_size(c.kv, keep), "cuda")
    abi.absp_evict(c.kv, w, keep, 1000, 7, c.d_table, w_out, kept[:keep].view(1, 1, keep), new, ws)
    assert abi.absp_check_device_error(ws) == (abi.ABSP_OK, 0)
    assert new.tolist() == [300]
    assert torch.equal(kept[:300], torch.arange(300, dtype=torch.int32, device="cuda"))
    for a in range(300, keep, 1 << 28):
        assert bool((kept[a:min(a + (1 << 28), keep)] == -1).all())
    assert int(kept[keep]) == 5
    assert torch.equal(w_out[..., :300], w[..., :300]) and bool((w_out[..., 300:] == -3.0).all())
    assert torch.equal(c.k.view(torch.int16), k.view(torch.int16))
    assert torch.equal(c.v.view(torch.int16), v.view(torch.int16))


# ------------------------------------------- the one-block selection's passes --

ONE_WARPS = 16


def _sampled(L):
    """Positions whose keys the one-block selection's first pass counts: the
    first of every four in the first 128 of every 512 of a warp's run."""
    run = -(-L // (128 * ONE_WARPS)) * 128
    p = np.arange(L)
    in_run = p % run
    return (in_run % 512 < 128) & (p % 4 == 0)


def _keys(w):
    u = (w + np.float32(0)).view(np.uint32)
    return np.where(u >> 31 != 0, ~u, u | np.uint32(0x80000000)).astype(np.int64)


def _sample_misses(w, L, keep, protect, recent):
    """Whether the threshold lies outside the range that the sample suggests."""
    mid = np.arange(protect, L - recent)
    left = keep - protect - recent
    k = _keys(w[:L])
    s = np.sort(k[mid][_sampled(L)[mid]] >> 21)[::-1]
    m = s.size
    at, d = m * left / mid.size, 2 * np.sqrt(m) + 8
    hi = (int(s[int(at - d) - 1]) << 21) + 0x1FFFFF if at > d + 1 else 1 << 40
    lo = int(s[int(at + d) - 1]) << 21 if int(at + d) <= m else 0
    threshold = np.sort(k[mid])[::-1][left - 1]
    return not lo <= threshold <= hi


def _check_evict(abi, c, w, dst, keep, protect, recent, alias):
    before, wo, kept, new = _run_evict(abi, c, w, dst, keep, protect, recent, alias, alias)
    k2, v2, wo2, kept2, new2 = CO.evict(w, c.lens, keep, protect, recent, before[0], before[1], c.table, dst,
                                        before[2])
    assert np.array_equal(kept, kept2) and np.array_equal(new, new2)
    assert np.array_equal(wo.view(np.int32), wo2.view(np.int32))
    assert np.array_equal(_bits(c.k), k2) and np.array_equal(_bits(c.v), v2)


@pytest.mark.parametrize("high", [True, False])
@pytest.mark.parametrize("where", ["fresh", "in_place"])
def test_evict_when_the_sample_misleads(abi, high, where):
    """Sampled positions hold the largest (smallest) weights: the threshold
    lies outside the range that they bound, and every key is counted again."""
    lens, keep, protect, recent = [6000, 4500, 300], 2500, 20, 100
    c, w, dst = _evict_case(abi, lens, 2, keep, protect, recent, where, "normal", seed=64)
    for s, L in enumerate(lens):
        w[s, :, :L][:, _sampled(L)] += 1000 if high else -1000
    for s in range(2):
        for h in range(2):
            assert _sample_misses(w[s, h], lens[s], keep, protect, recent)
    _check_evict(abi, c, w, dst, keep, protect, recent, where == "in_place")


@pytest.mark.parametrize("weights", ["normal", "ties", "odd", "misleading"])
def test_evict_keys_beyond_the_blocks_cache(abi, weights):
    """75 units of about 30,000 tokens: a block per unit, 24K keys of it in
    shared memory and the rest read again in every pass.  The sequences list
    the same source pages, as those of one prompt do."""
    S, P, keep, protect, recent = 75, 1900, 3000, 17, 400
    r = np.random.default_rng(65)
    lens = [P * 16 - 23 * s for s in range(S - 2)] + [2900, 24 * 1024 + 1]
    pk = -(-keep // 16)
    perm = r.permutation(P + S * pk).astype(np.int32)
    c = Case(abi, [1], 1, 1)
    c.lens, c.S, c.cap = lens, S, P * 16
    c.table = np.ascontiguousarray(np.broadcast_to(perm[:P], (S, P)))
    dst = perm[P:].reshape(S, pk)
    g = torch.Generator(device="cuda").manual_seed(66)
    c.k = torch.randn((P + S * pk, 1, 16, 128), generator=g, device="cuda").bfloat16()
    c.v = torch.randn((P + S * pk, 1, 16, 128), generator=g, device="cuda").bfloat16()
    c.d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    c.d_table = torch.from_numpy(c.table).cuda()
    c.kv = abi.LayerKV(c.d_lens, c.d_table, c.k, c.v, [16], 1)
    w = r.standard_normal((S, 1, c.cap)).astype(np.float32)
    if weights == "ties":
        w = np.round(2 * w)
    elif weights == "odd":
        w[r.random(w.shape) < 0.3] = np.nan
        w[r.random(w.shape) < 0.05] = np.inf
        w[r.random(w.shape) < 0.2] = -0.0
    elif weights == "misleading":
        for s, L in enumerate(lens):
            w[s, :, :L][:, _sampled(L)] -= 1000
        assert _sample_misses(w[0, 0], lens[0], keep, protect, recent)
    _check_evict(abi, c, w, dst, keep, protect, recent, False)
