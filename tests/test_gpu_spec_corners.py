"""Corners of the speculative-decoding operators on the GPU: steps larger than their capacity,
scores that are all NaN, paths cut short, lengths of the type's lowest value, the most requests."""
from __future__ import annotations

import numpy as np
import pytest

import oracle.speculative as ref
from gpu_common import announce, dev, to_dev
from test_gpu_spec import Case, raw, run_plan, tl, torch, values  # noqa: F401 (fixtures among them)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------- more tokens than the capacity
@pytest.mark.parametrize("R,block,tree", [(2, 16, True), (2, 16, False), (40, 16, True), (700, 32, True), (700, 64, False)])
def test_plan_beyond_capacity(tl, torch, R, block, tree):
    """Capacities below the step's tokens: at a request's border, inside one, at the first token, none at all."""
    rng = np.random.default_rng(R + block)
    new = rng.choice([0, 1, 5, 33, 64, 90], R)
    new[0] = 5
    ctx = rng.integers(0, 200, R)
    owned = np.maximum(-(-ctx // block) - (rng.random(R) < 0.2), 0)
    width = int((-(-(ctx + new) // block)).max())
    table = np.arange(R * width).reshape(R, width)
    free = np.arange(R * width, 2 * R * width)
    total = int(new.sum())
    for T in sorted({0, 1, 4, 5, 6, total // 2, int(new[:R // 2].sum()), total - 1, total}):
        announce(f"step_plan R={R} tokens={total} capacity={T}")
        parents = rng.integers(-1, 30, T) if tree else None
        run_plan(tl, torch, ctx, new, owned, table, free, 0, T, block, parents)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_step_beyond_capacity(tl, torch, e4m3, tree):
    """A request that does not fit the step's tokens is not served: nothing of what its pages held before
    is seen, no page is taken, nothing is committed; the requests before it are as they would be alone."""
    announce(f"a step beyond its capacity, e4m3={e4m3} tree={tree}")
    d, H, G, D, block, T = dev(), 2, 2, 128, 16, 10
    ctx, new, parents = [20, 30, 12], [5, 8, 3], [-1, 0, 0, 1, 1] + [-1, 0, 1, 2, 3]
    c = Case(tl, [(5, 20), (5, 33), (0, 12)], H, G, D, e4m3, block, tree=tree, seed=31)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=d)
    owned = [2, 2, 1]                                  # request 1 needs one page more
    free = np.setdiff1d(np.arange(c.pages), c.table[c.table < c.pages])
    table = i32(np.where(c.table < c.pages, c.table, 0))
    q_start, kv, slots, _, mask, owned_out, head = tl.step_plan(
        i32(ctx), i32(new), i32(owned), table, i32(free), i32([0]), T, block, parents=i32(parents) if tree else None)
    assert q_start.tolist() == [0, 5, 10, 10] and kv.tolist() == [25, 0, 0]
    assert owned_out.tolist() == owned and head.tolist() == [0] and (slots[5:] == -1).all()
    c.kv = np.array([25, 0, 0], dtype=np.int32)
    c.mask = mask.cpu().numpy().view(np.uint64) if tree else None
    c.call(block_table=table, q_start=q_start, kv_lens=kv).check(only=[0])
    assert (values(raw(c.out))[5:] == 0).all() and torch.isneginf(c.lse[5:]).all()
    done = tl.kv_commit(i32([1, 4, 1]), i32([[0, -1, -1, -1], [0, 1, 2, 4], [0, -1, -1, -1]]), i32(ctx), kv, table,
                        c.args["k_cache"], c.args["v_cache"], c.args["k_scale"], c.args["v_scale"])
    assert done.tolist() == [21, 30, 12]


# --------------------------------------------------------------------------- rows whose scores are all NaN
@pytest.mark.parametrize("D,e4m3,nodes,context", [(64, False, 3, 40), (128, False, 8, 100), (128, False, 16, 70),
                                                  (256, False, 20, 9), (64, True, 64, 300), (256, True, 12, 50),
                                                  (128, False, 2, 9000), (128, True, 40, 6000),
                                                  (128, False, 40, 3000), (256, False, 20, 3000)])
def test_attention_queries_that_are_nan(tl, D, e4m3, nodes, context):
    """A query with a NaN has a NaN result and a NaN lse, which -inf (nothing seen) is not; its neighbours have theirs."""
    c = Case(tl, [(nodes, context), (1, 0), (nodes, 0)], 1, 4, D, e4m3, 32, seed=D + nodes)
    bad = [(0, 1), (nodes - 1, 3), (nodes, 0), (nodes + 1, 2)]
    for t, h in bad:
        c.q[t, h, (7 * t) % D] = np.nan
    c.mask[nodes + 1 + nodes - 1] = 0                  # sees nothing: -inf, also with a NaN in its query
    c.q[-1, 1, 0] = np.nan
    c.call()
    c.q[-1, 1, 0] = 0.0                                # check() counts its bounds from q; this row is exactly 0 below
    c.check()
    lse, out = c.lse.cpu().numpy(), values(raw(c.out))
    nan = np.zeros(lse.shape, bool)
    for t, h in bad:
        nan[t, h] = True
    nan[-1] = False
    np.testing.assert_array_equal(np.isnan(lse), nan)
    np.testing.assert_array_equal(np.isnan(out).all(-1), nan)
    assert np.isneginf(lse[-1]).all() and (out[-1] == 0).all()


# --------------------------------------------------------------------------- commits
def commit(tl, torch, accepted, path, ctx, kv, block=16, D=64, H=2, e4m3=False, seed=0):
    """kv_commit against the moves of the plain definition; returns the new lengths."""
    d, rng, R = dev(), np.random.default_rng(seed), len(ctx)
    width = 12
    table = rng.permutation(R * width).reshape(R, width).astype(np.int32)
    path, i32 = np.array(path, dtype=np.int32), lambda a: to_dev(np.array(a, dtype=np.int32), d)
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k, v, ks, vs = tl.kv_cache(R * width, H, block, D, dtype=kind, device=d)
    for c in (k, v):
        c.view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 256, c.view(torch.uint8).shape, dtype=np.uint8)))
    before = [raw(c).copy() for c in (k, v)]
    got = tl.kv_commit(i32(accepted), to_dev(path, d), i32(ctx), i32(kv), to_dev(table, d), k, v, ks, vs)
    torch.cuda.synchronize()
    moves, want = ref.commit_moves(accepted, path, ctx, kv, table, R * width, block)
    for c, old, which in ((k, before[0], "k"), (v, before[1], "v")):
        at = ref.offsets(which, 1 if e4m3 else 2, block, D)
        new = old.copy().reshape(old.shape[:2] + (-1,))
        for _, pa, ta, pb, tb in moves:
            new[pb][..., at[tb]] = old.reshape(new.shape)[pa][..., at[ta]]
        np.testing.assert_array_equal(raw(c).reshape(new.shape), new)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    return got.tolist()


@pytest.mark.parametrize("e4m3", [False, True])
def test_commit_of_a_path_cut_short(tl, torch, e4m3):
    """Nodes past the path's width are not known, so they are not committed; a prompt needs no path."""
    announce(f"kv_commit, paths narrower than the accepted nodes, e4m3={e4m3}")
    path = [[0, 2, 3], [0, 1, 2], [0, 4, -1], [-1, -1, -1]]
    got = commit(tl, torch, [5, 3, 2, 100], path, [20, 31, 7, 9], [36, 40, 17, 109], e4m3=e4m3)
    assert got == [23, 34, 9, 109]


def test_commit_of_lengths_of_the_lowest_value(tl, torch):
    """Negative lengths count as 0, down to the type's lowest."""
    announce("kv_commit, lowest lengths")
    low = -2 ** 31
    got = commit(tl, torch, [3, 3, low, 2], [[0, 2, 3]] * 4, [5, low, 8, 40], [low, 9, 14, low + 3])
    assert got == [5, 3, 8, 40]


# --------------------------------------------------------------------------- the most requests
@pytest.mark.parametrize("D,e4m3,G,nodes,form", [(256, False, 5, 8, "bf16_share128"), (256, True, 5, 8, "e4m3_share128"),
                                                 (64, False, 5, 16, "bf16_share128"), (64, True, 3, 4, "e4m3_split16"),
                                                 (256, False, 2, 4, "bf16_split16")])
def test_attention_of_the_most_requests(tl, D, e4m3, G, nodes, form):
    """4096 requests, most of them without tokens, in forms whose prefix sums lie behind the largest LDS rings."""
    rng = np.random.default_rng(D + G)
    reqs = [(0, int(c)) for c in rng.choice([0, 0, 0, 9], 4096)]
    for r in [0, 1, 255, 256, 511, 512, 513, 2047, 4094, 4095] + rng.integers(0, 4096, 30).tolist():
        reqs[r] = (int(rng.integers(1, nodes + 1)), int(rng.integers(0, 90)))
    reqs[777] = (nodes, 2500)                          # one that several workgroups share
    c = Case(tl, reqs, 1, G, D, e4m3, 16, seed=D + G).call(max_nodes=nodes).check()
    assert tl.last_kernel_name() == "tree_attention_" + form


# --------------------------------------------------------------------------- lengths past the table
@pytest.mark.parametrize("D,e4m3,G,n,tree", [(64, False, 2, 6, True), (128, False, 4, 5, True), (128, False, 4, 16, True),
                                             (128, True, 4, 40, True), (256, False, 3, 12, True), (256, True, 5, 9, False),
                                             (64, True, 2, 100, False), (128, False, 3, 150, False)])
def test_attention_lengths_past_the_table(tl, D, e4m3, G, n, tree):
    """Positions that the table has no page for are not there, and move nothing: a request's own tokens are still
    the last n of its length, be they in the table or not."""
    c = Case(tl, [(n, 100), (n, 37), (1, 60)], 2, G, D, e4m3, 16, tree=tree, seed=41)
    width = (100 + n // 2) // 16                       # ends inside request 0's own tokens
    kernel = to_dev(c.table[:, :width].copy(), dev())
    c.table[:, width:] = -1                            # what the plain definition goes by
    c.call(block_table=kernel).check()
    # lengths of which not even the context fits, up to the type's largest
    c.kv[0] = 16 * width + n
    c.table = np.concatenate([c.table, np.full((3, -(-int(c.kv[0]) // 16)), -1, np.int32)], 1)
    c.call(block_table=kernel).check()
    out, lse = c.out.clone(), c.lse.clone()
    for far in (16 * width + n + 1, 1 << 30, (1 << 31) - 1):
        c.kv[0] = far
        c.call(block_table=kernel)
        assert c.out.equal(out) and c.lse.equal(lse), far
