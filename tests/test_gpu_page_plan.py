"""page_plan against the step written out request by request (cache4_ref.plan): whole numbers, so equal."""
import numpy as np
import pytest
import torch

import cache4_ref as ref
import kda_gated_delta_02_gb300 as kda

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def make(R, ctx_max, new_max, page, seed, over=2):
    r = np.random.default_rng(seed)
    ctx = r.integers(0, ctx_max + 1, R)
    new = r.integers(0, new_max + 1, R)
    held = -(-ctx // page) + (r.random(R) < 0.2)  # some keep a page more than their tokens fill
    total = np.maximum(held, -(-(ctx + new) // page))
    B = int(total.max()) + over
    pool = r.permutation(int(total.sum()) + 5)
    table = np.full((R, B), -7)
    at = 0
    for i in range(R):
        table[i, :held[i]] = pool[at:at + held[i]]
        at += int(held[i])
    return ctx, new, held, table, pool[at:].copy(), page


def check(ctx, new, held, table, free, page, T, count=None):
    count = len(free) if count is None else count
    t, st = dev(table), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kda.page_plan(dev(ctx), dev(new), dev(held), t, dev(free), dev([count]), page, T, status=st)
    want, status = ref.plan(ctx, new, held, table, free, count, page, T)
    for name, x in zip(("cu_seqlens", "seq_len", "slot_map", "positions", "page_count", "free_count"), got):
        assert x.dtype == torch.int32 and x.cpu().tolist() == list(map(int, want[name])), name
    assert np.array_equal(t.cpu().numpy(), want["table"])
    assert st.item() == status
    return got, status


@pytest.mark.parametrize("R,ctx,new,page", [(1, 0, 1, 16), (1, 4000, 1, 64), (3, 100, 700, 16), (256, 2000, 8, 64),
                                            (257, 500, 40, 128), (1024, 90, 9, 32), (1025, 90, 9, 16), (3001, 60, 5, 256),
                                            (7, 1, 20000, 32)])
def test_steps(R, ctx, new, page):
    c = make(R, ctx, new, page, seed=R + new)
    _, status = check(*c, T=int(c[1].sum()) + R % 3)
    assert status == 0


def test_no_new_tokens_and_no_rows():
    check(np.array([0, 5]), np.array([0, 0]), np.array([0, 1]), np.array([[-1], [3]]), np.array([0, 1, 2]), 16, T=0)
    check(np.array([0, 5]), np.array([0, 0]), np.array([0, 1]), np.array([[-1], [3]]), np.zeros(0, dtype=int), 16, T=4)


@pytest.mark.parametrize("R", [6, 700, 2100])
def test_pages_that_run_out(R):
    c = make(R, 50, 60, 16, seed=R)
    need = np.maximum(0, -(-(c[0] + c[1]) // 16) - c[2]).sum()
    for count in (0, int(need) // 2, int(need) - 1, int(need)):
        _, status = check(*c, T=int(c[1].sum()), count=count)
        assert status == (32 if count < need else 0)


def test_refused_requests():
    ctx, new, held, table, free, page = make(40, 100, 30, 16, seed=4)
    new[3], ctx[9], held[12], held[20] = -2, -1, -3, table.shape[1] + 1
    ctx[30] = table.shape[1] * page
    ctx[31], new[31] = 2 ** 31 - 1, 9
    _, status = check(ctx, new, held, table, free, page, T=int(np.maximum(new, 0).sum()))
    assert status == 1
    # rows that end past T
    c = make(10, 100, 30, 16, seed=5)
    _, status = check(*c, T=int(c[1].sum()) - 1)
    assert status == 1


def test_a_free_count_out_of_range_hands_out_nothing():
    ctx, new, held, table, free, page = make(5, 0, 9, 16, seed=6)
    new[:] = 5
    held[:] = 0
    for count in (-1, len(free) + 1):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = kda.page_plan(dev(ctx), dev(new), dev(held), dev(table), dev(free), dev([count]), page, 25, status=st)
        assert st.item() == kda.STATUS_NO_PAGES
        assert (got[2] == -1).all() and got[5].item() == count and (got[4] == 0).all()


def test_table_entries_that_are_not_pages():
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = kda.page_plan(dev([3, 3, 3]), dev([1, 1, 1]), dev([1, 1, 1]), dev([[-1], [2], [2 ** 30]]), dev([0]), dev([1]), 16, 3,
                        status=st)
    assert got[2].tolist() == [-1, 35, -1] and st.item() == kda.STATUS_BAD_PAGE


def test_steps_follow_one_another_in_a_graph():
    """Three decode steps by replays equal three calls; the counts are copied back between them."""
    ctx, new, held, table, free, page = make(12, 40, 0, 16, seed=8, over=5)
    R = len(ctx)
    free = np.concatenate([free, np.arange(1000, 1060)])

    def state():
        return [dev(ctx), dev(np.full(R, 13)), dev(held), dev(table), dev(free), dev([len(free)])]

    def step(s):
        got = kda.page_plan(*s[:4], s[4], s[5], page, R * 13)
        s[0].copy_(got[1])
        s[2].copy_(got[4])
        s[5].copy_(got[5])
        return got

    a, b = state(), state()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(state())
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(b)
    for _ in range(3):
        want = step(a)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got))
        assert torch.equal(a[3], b[3]) and torch.equal(a[5], b[5])
