"""pa_build_tables where a step's places, blocks or sequences run out, and loops of steps that go on from there."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from oracle import tree as otree  # noqa: E402
from test_gpu_tables import Server, compare, make, oracle_of, run  # noqa: E402
from tree_harness import Batch, check, random_parents  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [False, True])
def test_idle_sequences_behind_the_last_token_place(pa, cuda_device, tree):
    """Sequences whose tokens pass the arrays' end get nothing; idle ones behind them keep their contexts."""
    rng = np.random.default_rng(8)
    for S in (2, 20, 700):
        h = make(rng, S, 40, 0, 9, 16, tree, spare_blocks=4)
        h["new_lens"][0], h["new_lens"][-1] = 8, 0
        N = 4 if S == 2 else int(h["new_lens"].sum()) // 2
        if tree:
            h["parents"] = np.array([x for n in h["new_lens"] for x in random_parents(rng, int(n))], dtype=np.int32)
        want = oracle_of(h, N)
        assert want["context_lens"][-1] == h["context_lens"][-1] > 0 and 0 in want["context_lens"]
        compare(run(pa, cuda_device, h, N, 1), want, 1, f"S={S}")
        assert pa.pa_get_error() == pa.PA_DEVERR_QUERY


def test_no_sequences(pa, cuda_device):
    """An empty batch leaves no stale slot, position, start or list entry behind."""
    dev = cuda_device
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    empty = torch.empty(0, dtype=torch.int32, device=dev)
    for stream in (None, torch.cuda.Stream()):
        for tree in (False, True):
            slots = torch.full((9,), 5, dtype=torch.int64, device=dev)
            pos, starts, first = torch.full((9,), 5, dtype=torch.int32, device=dev), i32(7), i32(-9)
            par, mask = (i32(*[0] * 9), torch.full((9, 2), 5, dtype=torch.int64, device=dev)) if tree else (None, None)
            torch.cuda.synchronize()
            pa.pa_build_tables(empty.view(0, 4), empty, empty.clone(), starts, slots, pos, first, empty, empty, empty,
                               i32(1, 2, 3), i32(2), 16, 10, parents=par, tree_mask=mask, stream=stream)
            torch.cuda.synchronize()
            assert slots.tolist() == [-1] * 9 and pos.tolist() == [0] * 9 and starts.tolist() == [0]
            assert first.tolist() == [2] and (mask is None or not mask.any())


class KeepingServer(Server):
    """The loop of steps with pa_commit_tree's ``context_lens_before``; ``in_place``: the new lengths written over the
    old ones."""

    def __init__(self, *a, in_place, **kw):
        super().__init__(*a, **kw)
        self.in_place = in_place

    def step(self):
        pa = self.pa
        pa.pa_build_tables(self.bt, self.held2, self.ctx2, self.qs, self.slots, self.pos, self.first2, self.held,
                           self.ctx, self.new, self.free, self.first, 16, self.k.shape[0], parents=self.par,
                           tree_mask=self.mask)
        pa.pa_reshape_and_cache(self.nk, self.nv, self.k, self.v, self.slots)
        pa.pa_decode_tree(self.out, self.q, self.k, self.v, self.bt, self.ctx2, self.qs, self.mask, self.scale,
                          self.most, self.ws)
        kept = self.ctx if self.in_place else self.kept
        pa.pa_commit_tree([self.k], [self.v], self.bt, self.ctx2, self.qs, self.mask, self.acc, kept,
                          context_lens_before=self.ctx)
        self.held.copy_(self.held2)
        if not self.in_place:
            self.ctx.copy_(self.kept)
        self.first.copy_(self.first2)


def run_dry(server, steps, dry, replay, seed):
    """Random steps; in those of `dry` the free list is at its end. Every sequence's kept K/V, on the host, gives the
    reference of each step; the oracle says which sequences a step serves."""
    pa, rng = server.pa, np.random.default_rng(seed)
    S, H, G, d = server.S, server.H, server.G, server.d
    kept = [([], []) for _ in range(S)]
    unserved = 0
    for step in range(steps):
        new = rng.integers(0, server.most + 1, S) if step else rng.integers(1, server.most + 1, S)
        N = int(new.sum())
        parents = [random_parents(rng, int(n)) for n in new]
        acc = [int(rng.integers(-1, n)) if n else -1 for n in new]
        g = torch.Generator().manual_seed(1000 * seed + step)
        nk, nv = (torch.randn((N, G, d), generator=g).to(server.q.dtype) for _ in range(2))
        q = torch.randn((N, H, d), generator=g).to(server.q.dtype)
        server.new.copy_(torch.from_numpy(new.astype(np.int32)))
        server.acc.copy_(torch.tensor(acc, dtype=torch.int32))
        server.par[:N] = torch.tensor([x for p in parents for x in p], dtype=torch.int32)
        server.nk[:N], server.nv[:N], server.q[:N] = nk.to(server.dev), nv.to(server.dev), q.to(server.dev)
        server.out.fill_(7.0)
        at_first = server.first.clone()
        if step in dry:
            server.first.fill_(server.free.numel())
        plan = otree.build_tables(server.bt.cpu().numpy(), server.held.tolist(), [len(k[0]) for k in kept], new,
                                  server.free.tolist(), int(server.first), 16, server.N)
        replay()
        torch.cuda.synchronize()
        if step in dry:
            server.first.copy_(at_first)
        want = np.full((server.N, H, d), np.nan)
        at, short = 0, 0
        for s in range(S):
            n, served = int(new[s]), plan["context_lens"][s] == len(kept[s][0]) + new[s]
            seen = otree.ancestors(parents[s])
            for i in range(n):
                if not served:
                    want[at + i] = 0.0
                    continue
                rows = [at + j for j in range(n) if seen[i, j]]
                K = torch.stack(kept[s][0] + [nk[r] for r in rows]).double().numpy()
                V = torch.stack(kept[s][1] + [nv[r] for r in rows]).double().numpy()
                for h in range(H):
                    z = K[:, h // (H // G)] @ q[at + i, h].double().numpy() * server.scale
                    w = np.exp(z - z.max())
                    want[at + i, h] = w @ V[:, h // (H // G)] / w.sum()
            if served and acc[s] >= 0:
                for j in range(n):
                    if seen[acc[s], j]:
                        kept[s][0].append(nk[at + j])
                        kept[s][1].append(nv[at + j])
            short += not served
            at += n
        check(server.out, want, f"step {step}")
        assert bool((server.out[N:] == 7.0).all())
        assert server.ctx.tolist() == [len(k[0]) for k in kept], step
        assert pa.pa_get_error() == (pa.PA_DEVERR_NO_BLOCKS if short else 0)
        unserved += short
    assert unserved >= len(dry) and max(len(k[0]) for k in kept) > 16
    held, bt = server.held.tolist(), server.bt.cpu()
    used = [int(b) for i in range(S) for b in bt[i, :held[i]]]
    assert len(set(used)) == len(used) and min(used) >= 0
    for i in range(S):
        for t, row in enumerate(kept[i][0]):
            assert torch.equal(server.k[int(bt[i, t // 16]), :, t % 16].cpu(), row)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("heads", [(8, 2, 128, torch.bfloat16), (2, 2, 64, torch.float32)])
def test_a_loop_whose_free_list_runs_dry(pa, cuda_device, heads, graph, in_place):
    """Unserved sequences keep what they have cached, and the next step serves them."""
    H, G, d, dt = heads
    s = KeepingServer(pa, cuda_device, 5, H, G, d, 120, 20, 12, 3, dtype=dt, in_place=in_place)
    replay = s.step
    if graph:
        s.step()  # warm-up: no new tokens
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
        replay = g.replay
    run_dry(s, 10, (2, 5, 6), replay, 43)


@pytest.mark.parametrize("layers", [1, 150])
def test_commit_keeps_the_lengths_of_unserved_sequences(pa, cuda_device, layers):
    """Also with more layers than one launch takes, and with old lengths that cannot be."""
    b = Batch(63, [20, 3, 40, 7], [5, 4, 6, 2], 2, 2, 64, "f16")
    x = b.gpu(cuda_device)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=cuda_device)  # noqa: E731
    x.context_lens = i32(25, 0, 46, 0)
    acc = i32(-1, 2, -1, 1)
    pools = [x.k.clone() for _ in range(2 * layers)]
    for before, want in ((i32(20, 33, 40, 0), [20, 33, 40, 0]), (i32(9, 3, 9, -4), [20, 3, 40, 0])):
        for out in (before, i32(-9, -9, -9, -9)):
            keep = before.clone()
            pa.pa_commit_tree(pools[:layers], pools[layers:], x.block_tables, x.context_lens, x.query_starts, x.mask, acc,
                              out, context_lens_before=before)
            assert out.tolist() == want
            before.copy_(keep)
        pa.pa_commit_tree(pools[:layers], pools[layers:], x.block_tables, x.context_lens, x.query_starts, x.mask, acc, out)
        assert out.tolist() == [20, 0, 40, 0]
    assert all(torch.equal(p, x.k) for p in pools)
    assert pa.pa_get_error() == 0


@pytest.mark.parametrize("layout", ["HND", "NHD"])
def test_commit_skips_rows_of_blocks_outside_the_pool(pa, cuda_device, layout):
    """A path that moves rows in a block that cannot be: recorded, that sequence's rows stay, the others' move. A path
    that is in place moves nothing and records nothing."""
    b = Batch(64, [20, 18, 9], [6, 6, 6], 2, 2, 64, "f16", layout=layout)
    b.mask = torch.from_numpy(otree.pack_mask([[j in (0, 2, i) for j in range(6)] for _ in range(3) for i in range(6)], 1))
    acc = [5, 5, 5]
    good = b.block_tables.clone()
    (k, v), lens = otree.commit_tree([b.k.view(torch.int16).numpy(), b.v.view(torch.int16).numpy()], good,
                                     b.context_lens, b.query_starts, b.mask.numpy(), [5, -1, 5], 16, layout)
    x = b.gpu(cuda_device)
    x.block_tables[1, 1] = b.nb  # rows 18 .. 23 of the second sequence lie there
    out = torch.full((3,), -9, dtype=torch.int32, device=cuda_device)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=cuda_device)  # noqa: E731
    pa.pa_commit_tree([x.k], [x.v], x.block_tables, x.context_lens, x.query_starts, x.mask, i32(acc), out, layout=layout)
    assert pa.pa_get_error() == pa.PA_DEVERR_BLOCK_ID
    assert out.tolist() == [lens[0], 18 + 3, lens[2]] == [23, 21, 12]
    assert (x.k.cpu().view(torch.int16).numpy() == k).all() and (x.v.cpu().view(torch.int16).numpy() == v).all()
    x = b.gpu(cuda_device)
    x.block_tables[1, 1] = -1
    x.mask[6:12] = 1
    pa.pa_commit_tree([x.k], [x.v], x.block_tables, x.context_lens, x.query_starts, x.mask, i32(acc), out, layout=layout)
    assert pa.pa_get_error() == 0 and out.tolist() == [23, 19, 12]
    assert (x.k.cpu().view(torch.int16).numpy() == k).all() and (x.v.cpu().view(torch.int16).numpy() == v).all()
