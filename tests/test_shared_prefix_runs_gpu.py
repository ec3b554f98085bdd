"""The shared prefix over many token tiles, on the GPU: runs of several tiles
per CTA, runs that cross from one unit to the next, one to five row tiles,
maxima that grow inside a run, bad pages inside a run.

The fp64 oracle runs on the GPU (torch, from the definition) and holds every
output and weight to the element-wise bounds of oracle.cache_oracle; the first
test pins it to that oracle.  Every shape also has to give the same bits each
time: a copy that meets another warp's rows shows as a difference.
"""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as CO

pytestmark = pytest.mark.gpu

D, PAGE, TILE = 128, 16, 128


@pytest.fixture(scope="module")
def abi():
    from block_sparse_attention_kv_b200 import build
    build.build()
    from block_sparse_attention_kv_b200 import abi as m
    return m


def segments(prefix, S, G, Hkv):
    """The kernel's plan: per CTA, (unit, tiles, row tiles of the unit) of its run."""
    sms = min(torch.cuda.get_device_properties(0).multi_processor_count, 160)
    tiles, row_tiles = -(-prefix // TILE), -(-S * G // 128)
    units = (row_tiles + 1) // 2 * Hkv
    total = tiles * units
    ctas = min(sms, total)
    chunk = -(-total // ctas)
    runs = []
    for c in range(ctas):
        f, end, run = min(c * chunk, total), min((c + 1) * chunk, total), []
        while f < end:
            unit = f // tiles
            n = min(tiles - f % tiles, end - f)
            run.append((unit, n, min(2, row_tiles - 2 * (unit // Hkv))))
            f += n
        runs.append(run)
    return runs


class Batch:
    """Sequences over one shared prefix, each with a few tokens of its own
    (`short`: sequences that do not hold the prefix).  Page tables are wide
    enough that no call takes the one-launch path."""

    def __init__(self, abi, S, Hq, Hkv, prefix, own, short=(), grow=None, seed=0):
        r = np.random.default_rng(seed)
        lens = [prefix + int(x) for x in r.integers(0, own + 1, size=S)]
        lens[0] = prefix                                  # nothing of its own
        for i, n in enumerate(short):
            lens[1 + i] = n
        pre = prefix // PAGE
        P = max(600 if S * Hkv <= 160 else 1, pre + (own + PAGE - 1) // PAGE + 1)
        need = [-(-(n - prefix if n >= prefix else n) // PAGE) for n in lens]
        pages = pre + sum(need) + 3
        perm = r.permutation(pages).astype(np.int32)
        table = np.full((S, P), -1, np.int32)
        at = pre
        for s, n in enumerate(lens):
            first = pre if n >= prefix else 0
            table[s, :first] = perm[:first]
            table[s, first:first + need[s]] = perm[at:at + need[s]]
            at += need[s]
        g = torch.Generator(device="cuda").manual_seed(seed)
        k = torch.randn((pages, Hkv, PAGE, D), generator=g, device="cuda")
        v = torch.randn((pages, Hkv, PAGE, D), generator=g, device="cuda")
        q = torch.randn((S, Hq, D), generator=g, device="cuda")
        if grow:
            # a common direction of queries and keys: scores rise by 10 (log2
            # units) per token tile over `grow` tiles, then start over, so that
            # every run sees its maximum grow and its last tiles do not hide it
            u = torch.zeros(D, device="cuda")
            u[::2] = 1.0
            q += 1.5 * u
            ramp = 10 * ((torch.arange(prefix, device="cuda") // TILE) % grow + 1)
            # q . u is about 1.5 * 64: a key offset of c * u adds 96 c / sqrt(128) * log2(e)
            c = ramp / (96 / D ** 0.5 * 1.4427)
            rows = c.view(pre, 1, PAGE, 1) * u
            k[torch.from_numpy(perm[:pre]).long().cuda()] += rows
        self.lens, self.table, self.S, self.Hq, self.Hkv, self.prefix = lens, table, S, Hq, Hkv, prefix
        self.k, self.v, self.q = k.bfloat16(), v.bfloat16(), q.bfloat16()
        self.d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.d_table = torch.from_numpy(table).cuda()
        self.kv = abi.LayerKV(self.d_lens, self.d_table, self.k, self.v, [16] * Hkv, Hq)
        self.out = torch.full_like(self.q, 3.0)
        self.ws = abi.alloc_workspace(abi.absp_full_workspace_size(self.kv, prefix, True), "cuda")
        self.ws[256:].fill_(0xFF)
        self.abi = abi

    def run(self, w_in=None, w_out=None):
        self.abi.absp_shared_decode(self.kv, self.q, self.prefix, w_in, w_out, self.out, self.ws)

    def want(self, left_out=()):
        """(out, weights, out bound, weights bound): the formulas and bounds of
        oracle.cache_oracle.attention, tokens of the prefix pages `left_out`
        not attended to."""
        u, G = 2.0 ** -24, self.Hq // self.Hkv
        cap = self.table.shape[1] * PAGE
        out = torch.zeros((self.S, self.Hq, D), dtype=torch.float64, device="cuda")
        ob = torch.zeros_like(out)
        w = torch.zeros((self.S, self.Hkv, cap), dtype=torch.float64, device="cuda")
        wb = torch.zeros_like(w)
        for s, L in enumerate(self.lens):
            if L == 0:
                continue
            pre = self.prefix if L >= self.prefix else 0
            n = -(-L // PAGE)
            pg = torch.from_numpy(self.table[s, :n]).long().cuda()
            K = self.k[pg].double().transpose(0, 1).reshape(self.Hkv, -1, D)[:, :L]
            V = self.v[pg].double().transpose(0, 1).reshape(self.Hkv, -1, D)[:, :L]
            live = torch.ones(L, dtype=torch.bool, device="cuda")
            if pre:
                for p in left_out:
                    live[p * PAGE:(p + 1) * PAGE] = False
            q = self.q[s].double().view(self.Hkv, G, D)
            x = q @ K.transpose(1, 2) / D ** 0.5
            x = x.masked_fill(~live, float("-inf"))
            e = torch.exp(x - x.amax(-1, keepdim=True))
            p = e / e.sum(-1, keepdim=True)
            mag = (q.abs() @ K.abs().transpose(1, 2)).amax(-1, keepdim=True) / D ** 0.5
            top = x.masked_fill(~live, 0).abs().amax(-1, keepdim=True)
            rel = torch.expm1(2 * (32 * u * mag + 12 * u * top)) + 2.0 ** -20
            o, A = p @ V, p @ V.abs()
            bound = A * (rel + 2.0 ** -16 + (n + 64) * 4 * u)
            if pre:
                bound = bound + 2.0 ** -8 * (p[..., :pre] @ V[:, :pre].abs())
            out[s], ob[s] = o.view(-1, D), (bound + 2.0 ** -8 * (o.abs() + bound) + 1e-30).view(-1, D)
            w[s, :, :L] = p.sum(1)
            wb[s, :, :L] = (p * rel).sum(1) + (G + 4) * u * p.sum(1) + G * 2.0 ** -126
        return out, w, ob, wb

    def close(self, want, w_out=None, was=None):
        out, w, ob, wb = want
        got = self.out.double()
        assert torch.isfinite(got).all()
        bad = (got - out).abs() > ob
        assert not bad.any(), (bad.nonzero()[:5], (got - out).abs()[bad][:5], ob[bad][:5])
        if w_out is None:
            return
        for s, L in enumerate(self.lens):
            a = self.prefix if L >= self.prefix else 0
            x = was[s, :, a:L].double() + w[s, :, a:L]
            tol = wb[s, :, a:L] + 2.0 ** -24 * (x.abs() + wb[s, :, a:L])
            assert ((w_out[s, :, a:L].double() - x).abs() <= tol).all(), s
            assert torch.equal(w_out[s, :, :a], was[s, :, :a])
            assert torch.equal(w_out[s, :, L:], was[s, :, L:])


def test_the_gpu_oracle_is_the_oracle(abi):
    b = Batch(abi, 5, 8, 2, 160, 40, short=(30,), grow=2, seed=1)
    f = lambda t: t.float().cpu().numpy().astype(np.float64)  # noqa: E731
    for got, exp in zip(b.want(), CO.attention(f(b.q), f(b.k), f(b.v), b.table, b.lens, 160)):
        assert np.allclose(got.cpu().numpy(), exp, rtol=1e-9, atol=1e-300)


RUNS = [
    # S, Hq, Hkv, prefix, own tokens, shorter sequences
    (20, 32, 8, 6160, 40, ()),            # one row tile, its last 48 rows empty; a last tile of one page
    (9, 16, 8, 20016, 20, (700, 0)),      # runs of nine tiles: ring and page masks go round
    (40, 32, 8, 14464, 33, (1, 200)),     # two row tiles, the second with one warp of rows
    (56, 32, 8, 6160, 17, ()),            # the second with three
    (64, 32, 8, 8208, 16, ()),            # two whole row tiles
    (72, 16, 4, 6000, 50, (0,)),          # three row tiles: units of two and of one
    (39, 32, 2, 9904, 64, (31,)),         # five row tiles, 16 heads per KV head
    (320, 128, 8, 256, 20, (100,)),       # more units than SMs: units that one CTA holds whole
]


@pytest.mark.parametrize("S,Hq,Hkv,prefix,own,short", RUNS)
@pytest.mark.parametrize("grow", [None, 4])
def test_long_prefix(abi, S, Hq, Hkv, prefix, own, short, grow):
    runs = segments(prefix, S, Hq // Hkv, Hkv)
    assert max(n for run in runs for _, n, _ in run) > 1          # several tiles in a run
    assert any(len(run) > 1 for run in runs)                      # and a change of unit
    for seed in (3, 4):
        b = Batch(abi, S, Hq, Hkv, prefix, own, short, grow, seed)
        was = torch.rand((S, Hkv, b.table.shape[1] * PAGE), device="cuda")
        w = was.clone()
        b.run(w, w)
        assert abi.absp_check_device_error(b.ws) == (abi.ABSP_OK, 0)
        b.close(b.want(), w, was)
        first, fw = b.out.clone(), w.clone()
        for _ in range(20):
            b.out.fill_(5.0)
            w.copy_(was)
            b.run(w, w)
            assert torch.equal(b.out.view(torch.int16), first.view(torch.int16))
            assert torch.equal(w, fw)


def test_the_shapes_reach_every_form_of_a_run(abi):
    runs = [r for S, Hq, Hkv, prefix, *_ in RUNS for r in segments(prefix, S, Hq // Hkv, Hkv)]
    steps = {(a[2], b[2]) for r in runs for a, b in zip(r, r[1:])}
    assert {(1, 1), (2, 2), (2, 1)} <= steps                      # row tiles before and after a change of unit
    assert {n for r in runs for _, n, t in r if t == 1} >= {1, 2, 3, 9}
    assert max(sum(n for _, n, _ in r) for r in runs) > 8         # more than the page masks in flight


def test_bad_pages_inside_a_run_are_left_out(abi):
    b = Batch(abi, 40, 32, 8, 14464, 20, seed=9)
    for i, bad in enumerate([(0, 3, 4, 450, 903), tuple(range(64, 84))]):
        t = b.d_table.clone()
        for p in bad:
            b.d_table[:, p] = (1 << 20) if p % 2 else -7
        b.run()
        assert abi.absp_check_device_error(b.ws)[0] == abi.ABSP_ERR_DEVICE_FAULT
        b.close(b.want(left_out=bad))
        b.d_table.copy_(t)
    b.run()
    assert abi.absp_check_device_error(b.ws) == (abi.ABSP_OK, 0)
    b.close(b.want())
