"""The paged 4-bit cache on the GPU: rows in and out against the format's
definition, and attention against a 64-bit reference on the cache's own bytes,
with per-element bounds from the kernel's roundings (cache4_ref)."""
import itertools

import numpy as np
import pytest
import torch

import cache4_ref as ref
import kda_gated_delta_02_gb300 as kda

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device="cuda")


def to64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,d,page", [(1, 1, 64, 16), (77, 3, 128, 16), (300, 2, 64, 64), (130, 5, 128, 256)])
def test_rows_come_back_as_the_format_says(T, H, d, page, dtype):
    g = torch.Generator().manual_seed(T * 7 + d)
    P = -(-T // page) + 2
    k = (torch.randn(T, H, d, generator=g) * torch.exp(torch.randn(T, H, 1, generator=g) * 3)).to(DT[dtype])
    v = torch.randn(T, H, d, generator=g).to(DT[dtype])
    k[0] = 0
    v[T // 2, :, :16] = 1e-6  # scale underflows to zero
    k[T - 1, 0, 3] = 1e5      # saturates
    slots = torch.randperm(P * page, generator=g)[:T].to(torch.int32)
    slots[T // 3] = -1
    before = torch.randint(0, 255, (P, H, page * 9 * d // 8), generator=g, dtype=torch.uint8)
    cache, st = before.cuda(), status_word()
    kda.cache4_append(k.cuda(), v.cuda(), slots.cuda(), cache, page, status=st)
    ko, vo = kda.cache4_read(cache, slots.cuda(), page, d, dtype=DT[dtype], status=st)
    assert st.item() == 0
    keep = (slots >= 0).numpy()
    for got, x in ((ko, k), (vo, v)):
        want = ref.held(x.float().numpy()) * keep[:, None, None]
        # six significant bits and exponents from -10 to 11: exact in every type
        assert np.array_equal(to64(got), want)
    # the bytes, through the reference's own reading of the layout
    dk, dv = ref.decode(cache.cpu().numpy(), d)
    at = slots.numpy()[keep]
    assert np.array_equal(dk[at // page, :, at % page], ref.held(k.float().numpy())[keep])
    assert np.array_equal(dv[at // page, :, at % page], ref.held(v.float().numpy())[keep])
    # no byte of another slot changed
    other = np.setdiff1d(np.arange(P * page), at)
    raw = lambda c: c.cpu().numpy().reshape(P, H, page // 16, ref.block_bytes(d))
    a, b = raw(before), raw(cache)
    ka, kb = 16 * d // 2, 16 * d // 16
    for p, o in zip(other // page, other % page):
        blk, tok = o // 16, o % 16
        pieces = [slice(tok * d // 2, (tok + 1) * d // 2), slice(ka + tok * d // 16, ka + (tok + 1) * d // 16)]
        pieces += [slice(ka + kb + grp * 128 + tok * 8, ka + kb + grp * 128 + tok * 8 + 8) for grp in range(d // 16)]
        pieces += [slice(2 * ka + kb + grp * 16 + tok, 2 * ka + kb + grp * 16 + tok + 1) for grp in range(d // 16)]
        for s in pieces:
            assert np.array_equal(a[p, :, blk, s], b[p, :, blk, s])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounding_at_every_tie(dtype):
    """Rows whose largest element sets the scale to every mantissa of e4m3 (ties of max / 6 among them) and whose other
    elements sit on and next to every midpoint of the codes."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    rows = []
    for e in (-9, -7, -6, 0, 3, 8):
        for m in np.arange(16, 32) / 16:  # halves of a scale step: ties of the scale itself
            s = m * 2.0 ** e
            near = [x * s * f for x in mids for f in (1.0, 1 + 2.0 ** -7)]
            rows.append([6 * s] + [x * (-1) ** i for i, x in enumerate(near)] + [0.0])
    x = torch.tensor(rows, dtype=torch.float64).to(DT[dtype])
    x = x.reshape(-1, 1, 16).repeat(1, 1, 4)  # d = 64
    T, page = x.shape[0], 16
    cache = kda.cache4_alloc(-(-T // page), 1, page, 64)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kda.cache4_append(x.cuda(), (-x).cuda(), slots, cache, page)
    k, v = kda.cache4_read(cache, slots, page, 64, dtype=DT[dtype])
    want = ref.held(x.float().numpy())
    assert np.array_equal(to64(k), want) and np.array_equal(to64(v), -want)


def test_rows_of_a_fused_projection_and_head_scales():
    T, Hq, H, d, page = 53, 4, 2, 128, 32
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T, (Hq + 2 * H) * d, generator=g).bfloat16().cuda()
    k = qkv[:, Hq * d:(Hq + H) * d].view(T, H, d)
    v = qkv[:, (Hq + H) * d:].view(T, H, d)
    ks, vs = torch.tensor([0.25, 8.0], device="cuda"), torch.tensor([2.0 ** -6, 1.0], device="cuda")
    cache = kda.cache4_alloc(2, H, page, d)
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kda.cache4_append(k, v, slots, cache, page, k_scale=ks, v_scale=vs)
    ko, vo = kda.cache4_read(cache, slots, page, d, dtype=torch.float32, k_scale=ks, v_scale=vs)
    assert np.array_equal(to64(ko), ref.held(k.float().cpu().numpy(), ks.cpu().numpy()))
    assert np.array_equal(to64(vo), ref.held(v.float().cpu().numpy(), vs.cpu().numpy()))


@pytest.mark.parametrize("where,what", [("k", float("nan")), ("v", float("inf")), ("k", float("-inf")), ("v", float("nan"))])
def test_rows_that_are_not_finite_are_marked(where, what):
    T, H, d, page = 20, 2, 64, 16
    x = {n: torch.randn(T, H, d).bfloat16() for n in "kv"}
    x[where][7, 1, 50] = what
    cache, st = kda.cache4_alloc(2, H, page, d), status_word()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    kda.cache4_append(x["k"].cuda(), x["v"].cuda(), slots, cache, page, status=st)
    assert st.item() == kda.STATUS_NOT_FINITE
    k, v = kda.cache4_read(cache, slots, page, d, dtype=torch.float32)
    marked = torch.zeros(T, H, dtype=torch.bool)
    marked[7, 1] = True
    for t in (k, v):
        assert torch.equal(t.isnan().all(-1).cpu(), marked) and torch.equal(t.isnan().any(-1).cpu(), marked)


def test_slots_past_the_cache_are_refused():
    T, H, d, page = 6, 1, 64, 16
    x = torch.ones(T, H, d, device="cuda").bfloat16()
    cache, st = kda.cache4_alloc(1, H, page, d), status_word()
    slots = dev([0, 16, 15, -1, 2 ** 31 - 1, -5])
    kda.cache4_append(x, x, slots, cache, page, status=st)
    assert st.item() == kda.STATUS_BAD_PAGE
    st.zero_()
    k, _ = kda.cache4_read(cache, slots, page, d, status=st)
    assert st.item() == kda.STATUS_BAD_PAGE
    one = ref.held(np.ones((1, 1, 64)))[0, 0, 0]  # 1 / 6 is not an e4m3 number
    assert k[:, 0, 0].tolist() == [one, 0, one, 0, 0, 0]


# ------------------------------------------------------------------ attention
class Case:
    """A cache with requests of the given lengths on shuffled pages; what no request holds has random bytes, NaN scales
    among them."""

    def __init__(self, lengths, new, Hq, H, d, page, dtype="bf16", seed=0, gain=1.0, ks=None, vs=None, extra_pages=3):
        g = torch.Generator().manual_seed(seed)
        self.page, self.d, self.lengths, self.new = page, d, lengths, new
        pages = [-(-n // page) for n in lengths]
        P, B = sum(pages) + extra_pages, max(max(pages), 1) + 1
        perm = torch.randperm(P, generator=g).numpy()
        self.table = np.full((len(lengths), B), -1, dtype=np.int64)
        at, slots = 0, []
        for r, n in enumerate(pages):
            self.table[r, :n] = perm[at:at + n]
            at += n
            p = np.arange(lengths[r])
            slots.append(self.table[r, p // page] * page + p % page if lengths[r] else np.zeros(0, dtype=np.int64))
        slots = np.concatenate(slots)
        total = len(slots)
        self.k = torch.randn(total, H, d, generator=g) * torch.exp(0.5 * torch.randn(1, H, d, generator=g))
        self.v = torch.randn(total, H, d, generator=g)
        self.ks = None if ks is None else dev(ks, torch.float32)
        self.vs = None if vs is None else dev(vs, torch.float32)
        raw = torch.randint(0, 256, (P, H, page * 9 * d // 8), generator=g, dtype=torch.uint8)
        raw[:, :, ::5] = 0x7F
        self.cache = raw.cuda()
        self.slots = dev(slots)
        if total:
            kda.cache4_append(self.k.bfloat16().cuda(), self.v.bfloat16().cuda(), self.slots, self.cache, page,
                              k_scale=self.ks, v_scale=self.vs)
        self.cu = np.concatenate(([0], np.cumsum(new)))
        self.q = (gain * torch.randn(int(self.cu[-1]), Hq, d, generator=g)).to(DT[dtype])
        self.args = (self.cache, dev(self.table), dev(lengths), dev(self.cu), page)

    def run(self, q=None, **kw):
        return kda.cache4_attention((self.q if q is None else q).cuda(), *self.args, k_scale=self.ks, v_scale=self.vs, **kw)

    def want(self, scale=None, window=0):
        k, v = ref.decode(self.cache.cpu().numpy(), self.d)
        k = k * (1 if self.ks is None else self.ks.cpu().double().numpy()[:, None, None])
        v = v * (1 if self.vs is None else self.vs.cpu().double().numpy()[:, None, None])
        return ref.attention(to64(self.q), k, v, self.table, self.lengths, self.cu, self.page,
                             self.d ** -0.5 if scale is None else scale, window)

    def check(self, scale=None, window=0, **kw):
        st = status_word()
        o, lse = self.run(scale=scale, window=window, return_lse=True, status=st, **kw)
        assert st.item() == 0
        want = self.want(scale, window)
        bo, bl = ref.attention_bounds(*want, bf16=self.q.dtype == torch.bfloat16)
        assert np.all(np.isfinite(to64(o)))
        assert np.all(np.abs(to64(o) - want[0]) <= bo), float(np.max(np.abs(to64(o) - want[0]) / bo))
        none = np.isneginf(want[1])
        got = to64(lse)
        assert np.array_equal(np.isneginf(got), none) and np.all(to64(o)[none] == 0)
        assert np.all(np.abs(got[~none] - want[1][~none]) <= bl[~none])
        return o, lse


EDGE = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,H,d,page", [(8, 1, 128, 64), (6, 2, 64, 16), (3, 3, 128, 16), (24, 2, 128, 32),
                                         (16, 1, 64, 256), (40, 2, 64, 128), (34, 1, 128, 64)])
def test_single_tokens_at_every_edge_length(Hq, H, d, page, dtype):
    lengths = [n for n in EDGE if n > 0]
    Case(lengths, [1] * len(lengths), Hq, H, d, page, dtype, seed=Hq + d).check(max_new=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 1, 7, 40])
@pytest.mark.parametrize("Hq,H,d,page", [(8, 1, 128, 64), (4, 2, 64, 16), (12, 1, 128, 16)])
def test_ragged_windows_of_queries(Hq, H, d, page, window, dtype):
    """Several queries per request: some more than the cache holds (those see nothing), requests without queries and
    without keys among them."""
    lengths = [0, 5, 1, 40, 97, 0, 130, 64]
    new = [0, 8, 3, 8, 1, 4, 7, 0]
    Case(lengths, new, Hq, H, d, page, dtype, seed=window).check(window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("Hq,H,d,page,n,L", [(8, 2, 128, 64, 70, 200), (3, 1, 64, 16, 129, 129), (5, 1, 128, 32, 61, 333),
                                             (1, 1, 64, 128, 200, 260)])
def test_prompt_chunks(Hq, H, d, page, n, L, window, dtype):
    Case([L, 33, L + 7], [n, 33, 2], Hq, H, d, page, dtype, seed=n).check(window=window, max_new=n)


def test_one_long_request_is_joined_from_its_shares():
    Case([20011], [1], 8, 1, 64, 64, seed=5).check(max_new=1)
    Case([9001, 17], [8, 8], 8, 2, 64, 16, seed=6).check(max_new=8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales_and_sharp_and_flat_maps(dtype):
    c = Case([150, 33], [3, 1], 8, 2, 128, 32, dtype, seed=9, ks=[0.5, 4.0], vs=[2.0 ** -8, 1.0])
    c.check()
    c.check(scale=0.0)
    c.check(scale=-0.3)
    Case([150], [2], 4, 1, 128, 16, dtype, seed=10, gain=30.0).check()      # one key takes almost all
    Case([150], [2], 4, 1, 128, 16, dtype, seed=11, gain=2.0 ** -40).check()  # queries far below one


def test_an_upper_bound_that_is_too_low_still_gives_every_query():
    Case([90, 12], [40, 2], 4, 1, 128, 64, seed=12).check(max_new=1)


def test_queries_of_a_fused_projection_and_given_buffers():
    c = Case([70, 9], [5, 2], 4, 2, 64, 16, seed=13)
    o, lse = c.check()
    wide = torch.randn(7, 4 * 64 + 96).bfloat16().cuda()
    wide[:, 32:32 + 256] = c.q.cuda().view(7, 256)
    view = wide[:, 32:32 + 256].view(7, 4, 64)
    out, l2 = torch.full((9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((9, 4), 7.0, device="cuda")
    kda.cache4_attention(view, *c.args, out=out[1:8], lse=l2[1:8], return_lse=True)
    assert torch.equal(out[1:8], o) and torch.equal(l2[1:8], lse)
    assert (out[[0, 8]] == 7).all() and (l2[[0, 8]] == 7).all()


def test_rows_past_the_last_request_are_not_touched():
    c = Case([40, 9], [2, 1], 8, 1, 128, 16, seed=14)
    q = torch.cat((c.q, torch.full((4, 8, 128), float("nan"), dtype=torch.bfloat16)))
    out = torch.full((7, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(q=q, out=out, max_new=2)
    assert torch.equal(out[:3], c.run(max_new=2)) and (out[3:] == 3).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 60])
def test_a_marked_token_reaches_only_queries_that_see_it(n, dtype):
    """A key or value that is not finite sits at a position that the last queries see and the first do not, next to
    keys of the same tile that all see."""
    L, H, page, d = 80, 2, 16, 128
    c = Case([L], [n], 4, H, d, page, dtype, seed=15)
    clean = c.run()
    pos = L - 2
    x = torch.randn(1, H, d)
    x[0, 1, 5] = float("inf")
    kda.cache4_append(c.k[pos:pos + 1].bfloat16().cuda(), x.bfloat16().cuda(), c.slots[pos:pos + 1], c.cache, page)
    o, lse = c.run(return_lse=True)
    sees = torch.zeros(n, 4, dtype=torch.bool)
    sees[n - 2:, 2:] = True  # the head with the mark, positions L - 2 and L - 1
    assert torch.equal(o.isnan().all(-1).cpu(), sees) and torch.equal(o.isnan().any(-1).cpu(), sees)
    assert torch.equal(lse.isnan().cpu(), sees)
    assert torch.equal(o[:n - 2], clean[:n - 2])


@pytest.mark.parametrize("n", [4, 40])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_queries_that_are_not_finite_stay_alone(n, what):
    c = Case([50, 20], [n, 1], 4, 1, 64, 16, seed=16)
    clean = c.run(max_new=n)
    q = c.q.clone()
    q[1, 2, 3] = what
    o = c.run(q=q, max_new=n)
    assert o[1, 2].isnan().all()
    o[1, 2] = clean[1, 2]
    assert torch.equal(o, clean)


@pytest.mark.parametrize("new", [1, 8, 50])
def test_the_same_call_gives_the_same_bits(new):
    c = Case([3000, 70, 500], [new] * 3, 16, 2, 128, 32, seed=17)
    a = c.run(return_lse=True)
    for _ in range(3):
        b = c.run(return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_another_stream_and_a_graph():
    c = Case([700, 33], [2, 1], 8, 2, 128, 64, seed=18)
    want = c.run()
    q, args = c.q.cuda(), c.args
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.cache4_attention(q, *args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(got)
    with torch.cuda.stream(s):
        kda.cache4_attention(q, *args, out=out)
        graph = torch.cuda.CUDAGraph()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            kda.cache4_attention(q, *args, out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("new", [1, 40])
def test_pages_past_4_gib(new):
    """Byte offsets of the pages need 64 bits."""
    H, d, page = 4, 128, 64
    P = (5 << 30) // (H * page * 9 * d // 8)
    cache = kda.cache4_alloc(P, H, page, d)
    L = 150
    table = dev([[P - 1, 1, P - 2]])
    pos = torch.arange(L, device="cuda")
    slots = (table[0, pos // page] * page + pos % page).int()
    k, v = torch.randn(2, L, H, d, device="cuda").bfloat16().unbind(0)
    kda.cache4_append(k, v, slots, cache, page)
    ko, _ = kda.cache4_read(cache, slots, page, d, dtype=torch.float32)
    assert np.array_equal(to64(ko), ref.held(k.float().cpu().numpy()))
    q = torch.randn(new, 8, d, device="cuda").bfloat16()
    o = kda.cache4_attention(q, cache, table, dev([L]), dev([0, new]), page)
    small = cache[[P - 1, 1, P - 2]].contiguous()
    assert torch.equal(o, kda.cache4_attention(q, small, dev([[0, 1, 2]]), dev([L]), dev([0, new]), page))


def near(a, b):
    """Two results whose shares of the keys were cut differently: each within half a bf16 step (2^-8) and the weights'
    rounding (2^-11 of the weighted |v|, here below four times the largest output) of the exact one."""
    return bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -8 * b.abs().max()).all())


@pytest.mark.parametrize("new", [1, 40])
def test_bad_lengths_and_pages_are_refused(new):
    c = Case([60, 60, 60], [new] * 3, 8, 1, 64, 16, seed=19)
    want = c.run()
    cache, table, lengths, cu, page = c.args
    st, out = status_word(), torch.full_like(want, 5.0)
    bad = lengths.clone()
    bad[1] = table.shape[1] * page + 1
    kda.cache4_attention(c.q.cuda(), cache, table, bad, cu, page, out=out, status=st)
    assert st.item() == kda.STATUS_BAD_SEQLENS
    assert near(out[:new], want[:new]) and near(out[2 * new:], want[2 * new:]) and (out[new:2 * new] == 5).all()
    for cut in ([0, new, 3 * new + 1, 3 * new], [0, new, -1, 3 * new]):  # queries past the end, and before the start
        st.zero_()
        out.fill_(5.0)
        kda.cache4_attention(c.q.cuda(), cache, table, lengths, dev(cut), page, out=out, status=st)
        assert st.item() == kda.STATUS_BAD_SEQLENS and near(out[:new], want[:new])
    for entry in (-1, cache.shape[0], 2 ** 31 - 1):
        st.zero_()
        t2 = table.clone()
        t2[1, 1] = entry
        o = kda.cache4_attention(c.q.cuda(), cache, t2, lengths, cu, page, status=st)
        assert st.item() == kda.STATUS_BAD_PAGE
        assert torch.equal(o[:new], want[:new]) and torch.equal(o[2 * new:], want[2 * new:])


@pytest.mark.parametrize("window", [0, 33])
def test_batches_of_single_tokens_and_chunks(window):
    """Requests of few rows and of many in one call, through both kernels, in every order of sizes."""
    lengths = [70, 300, 1, 129, 500, 64, 200, 31]
    new = [1, 40, 1, 3, 200, 1, 9, 4]
    for Hq, H, d, page in ((8, 1, 128, 64), (12, 4, 64, 16), (5, 1, 64, 32)):
        c = Case(lengths, new, Hq, H, d, page, seed=Hq + window)
        c.check(window=window)
        c.check(window=window, max_new=200)
        c.check(window=window, max_new=5)  # too low a bound picks another split, not another result


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_on_16_byte_boundaries(dtype):
    """Rows that are 16-byte but not 32-byte aligned (the wide accesses need 32)."""
    T, H, d, page = 37, 3, 64, 16
    step = 8 if dtype == "bf16" else 4
    g = torch.Generator().manual_seed(21)
    wide = torch.randn(T, 2 * H * d + step, generator=g).to(DT[dtype]).cuda()
    k, v = wide[:, step:step + H * d].view(T, H, d), wide[:, step + H * d:].view(T, H, d)
    cache, slots = kda.cache4_alloc(3, H, page, d), torch.arange(T, dtype=torch.int32, device="cuda")
    kda.cache4_append(k, v, slots, cache, page)
    ko, vo = kda.cache4_read(cache, slots, page, d, dtype=DT[dtype])
    assert np.array_equal(to64(ko), ref.held(k.float().cpu().numpy()))
    assert np.array_equal(to64(vo), ref.held(v.float().cpu().numpy()))
    # read into outputs on 16-byte boundaries, through the C ABI
    lib, n = kda.load_library(), T * H * d
    out = torch.zeros(2 * n + 3 * step, dtype=DT[dtype], device="cuda")
    po, at = out[step:step + n], out[2 * step + n:2 * step + 2 * n]
    assert lib.kda_cache4_read(cache.data_ptr(), slots.data_ptr(), T, H, d, 3, page, None, None, 0 if dtype == "bf16" else 1,
                               po.data_ptr(), at.data_ptr(), None, kda._stream(None)) == 0
    assert torch.equal(po.view(T, H, d), ko) and torch.equal(at.view(T, H, d), vo)
    assert (out[:step] == 0).all() and (out[step + n:2 * step + n] == 0).all() and (out[2 * step + 2 * n:] == 0).all()


@pytest.mark.parametrize("new", [1, 12, 50])
def test_nothing_is_written_outside_the_outputs(new):
    """Cache, outputs and workspace lie between bands of a sentinel byte."""
    def guarded(like, pad=4096):
        whole = torch.full((like.nbytes + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
        view = whole[pad:pad + like.nbytes].view(like.dtype).view(like.shape)
        view.copy_(like)
        return whole, view

    def intact(whole, pad=4096):
        return bool((whole[:pad] == 0xA5).all() and (whole[-pad:] == 0xA5).all())

    c = Case([400, 33, 90], [new] * 3, 8, 2, 128, 16, seed=23, extra_pages=0)
    want = c.run(return_lse=True)
    w_cache, cache = guarded(c.cache)
    kda.cache4_append(c.k.bfloat16().cuda(), c.v.bfloat16().cuda(), c.slots, cache, 16)
    assert intact(w_cache) and torch.equal(cache, c.cache)
    w_out, out = guarded(torch.zeros_like(want[0]))
    w_lse, lse = guarded(torch.zeros_like(want[1]))
    need = kda.cache4_attention_workspace_size(3, 3 * new, 8, 2, 128)
    w_ws, ws = guarded(torch.zeros(need, dtype=torch.uint8, device="cuda"))
    kda.cache4_attention(c.q.cuda(), cache, *c.args[1:], out=out, lse=lse, return_lse=True, workspace=ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert intact(w_out) and intact(w_lse) and intact(w_ws) and intact(w_cache)


@pytest.mark.parametrize("new", [1, 40])
def test_a_wait_that_runs_out_is_reported(new):
    """A build whose first wait gives up at once (copies, or products, in flight): the call sets KDA_STATUS_TIMEOUT and
    returns, the stream completes, and the ordinary library is right on the same inputs afterwards."""
    import ctypes

    from kda_gated_delta_02_gb300 import build
    test_lib, main = ctypes.CDLL(build.build_variant("shortwait", ["KDA_TEST_SHORT_FIRST_WAIT"])), kda.load_library()
    f = test_lib.kda_cache4_attention
    f.restype, f.argtypes = main.kda_cache4_attention.restype, main.kda_cache4_attention.argtypes
    c = Case([900, 300], [new, new], 8, 2, 128, 16, seed=24)
    cache, table, lengths, cu, page = c.args
    q, st = c.q.cuda(), status_word()
    out = torch.zeros_like(q)
    ws = torch.empty(kda.cache4_attention_workspace_size(2, 2 * new, 8, 2, 128), dtype=torch.uint8, device="cuda")
    assert f(q.data_ptr(), cache.data_ptr(), table.data_ptr(), lengths.data_ptr(), cu.data_ptr(), 2, 2 * new, 8, 2, 128,
             cache.shape[0], page, table.shape[1], new, 0, 128 ** -0.5, 8 * 128, None, None, out.data_ptr(), None, 0,
             ws.data_ptr(), ws.nbytes, st.data_ptr(), kda._stream(None)) == 0
    torch.cuda.synchronize()
    assert st.item() & kda.STATUS_TIMEOUT
    c.check(max_new=new)


@pytest.mark.parametrize("Hq,H,d", [(16, 1, 128), (17, 1, 64), (34, 2, 128), (48, 1, 64)])
def test_ragged_batches_at_the_widest_group_of_few_rows(Hq, H, d):
    """Single tokens, none and several beside one another, where a group's heads are as many as the few-row kernel takes,
    and more."""
    Case([70, 40, 300, 1, 129], [1, 0, 8, 1, 2], Hq, H, d, 32, seed=Hq).check(max_new=8)


def test_calls_in_a_row_on_one_workspace():
    """Kernels of a call start while its others end; those of the next call on the same workspace do not."""
    cases = [Case([900, 64, 300, 2000, 33], [1, 40, 1, 5, 2], 8, 1, 128, 64, seed=31),
             Case([129, 1500, 40, 700], [100, 1, 1, 300], 8, 1, 128, 64, seed=32)]
    alone = [c.run() for c in cases]
    R, T = 5, max(c.q.shape[0] for c in cases)
    ws = torch.empty(kda.cache4_attention_workspace_size(R, T, 8, 1, 128), dtype=torch.uint8, device="cuda")
    q = [c.q.cuda() for c in cases]
    outs = [[torch.empty_like(x) for x in q] for _ in range(10)]
    torch.cuda.synchronize()
    for o in outs:
        for c, x, out in zip(cases, q, o):
            kda.cache4_attention(x, *c.args, out=out, workspace=ws)
    for o in outs:
        for a, b in zip(o, alone):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("power", [15, 20, 21, 24, 40])
@pytest.mark.parametrize("lengths,new,Hq,H,d", [([150, 33, 7000], [1, 3, 1], 8, 2, 128), ([300, 20], [40, 20], 2, 1, 64),
                                                ([333, 9000], [90, 40], 6, 2, 128)])
def test_scores_far_apart(lengths, new, Hq, H, d, power, dtype):
    """Scores of 2^power and more: one key takes all where the next is further away than the scores' rounding, the output
    is then its value (the weight's rounding to f16 for bf16 calls, then the output's own), and every row is finite and
    no larger than the largest value."""
    c = Case(lengths, new, Hq, H, d, 32, dtype, seed=power + d, gain=2.0 ** power)
    o, lse = c.run(return_lse=True, max_new=max(new))
    keys, values = ref.decode(c.cache.cpu().numpy(), d)
    want, want_lse, _, _, top = c.want()
    o, lse, q, G, clear = to64(o), to64(lse), to64(c.q), Hq // H, 0
    assert np.isfinite(o).all() and np.isfinite(lse).all()
    err = top * 2.0 ** -17  # of a score (cache4_ref.attention_bounds)
    assert np.all(np.abs(lse - want_lse) <= err + 2.0 ** -19 * (1 + np.abs(want_lse)))
    rel = 2.0 ** -8 + 2.0 ** -11 if dtype == "bf16" else 2.0 ** -19
    for r, (n, L) in enumerate(zip(new, lengths)):
        pages = c.table[r, :-(-L // 32)]
        for h in range(H):
            k, v = (t[pages, h].reshape(-1, d)[:L] for t in (keys, values))
            largest = np.maximum.accumulate(np.abs(v))
            for i, x in itertools.product(range(n), range(h * G, h * G + G)):
                row, sees = c.cu[r] + i, L - n + i + 1
                s = k[:sees] @ q[row, x] * d ** -0.5
                assert np.all(np.abs(o[row, x]) <= (1 + rel) * largest[sees - 1])
                first, second = np.argmax(s), np.sort(s)[-2] if sees > 1 else -np.inf
                if s[first] - second > 4 * err[row, x] + 40:  # e^-40 is below f16's smallest weight
                    clear += 1
                    assert np.all(np.abs(o[row, x] - v[first]) <= rel * np.abs(v[first]) + 2.0 ** -30)
    assert clear > 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 40, 200])
def test_scales_that_are_not_finite_are_seen(n, dtype):
    """A scale of NaN, or a head's key scale: every row that sees a key is NaN there, and a row that sees none is zero."""
    c = Case([90, 260], [100, n], 4, 2, 64, 16, dtype, seed=41)
    seen = torch.ones(100 + n, dtype=torch.bool)
    seen[:10] = False  # 90 keys, 100 queries
    o, lse = c.run(return_lse=True, scale=float("nan"))
    assert o[seen].isnan().all() and lse[seen].isnan().all()
    assert (o[~seen] == 0).all() and torch.isneginf(lse[~seen]).all()
    o = c.run(scale=float("inf"))
    assert o[seen].isnan().all() and (o[~seen] == 0).all()
    clean = c.run()
    c.ks = dev([1.0, float("nan")], torch.float32)
    o, lse = c.run(return_lse=True)
    assert o[seen][:, 2:].isnan().all() and lse[seen][:, 2:].isnan().all()
    assert torch.equal(o[:, :2], clean[:, :2]) and (o[~seen] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,new", [([1, 40], [1, 2]), ([5000], [1]), ([100, 6000], [40, 30]), ([500], [300])])
def test_scores_of_minus_infinity_alone_are_not_an_empty_row(lengths, new, dtype):
    """A query whose scores are all -inf has o = 0 / 0, not the zero of a query that sees nothing."""
    c = Case(lengths, new, 4, 2, 64, 16, dtype, seed=42)
    c.k[:, :, 5] = -3.0
    kda.cache4_append(c.k.bfloat16().cuda(), c.v.bfloat16().cuda(), c.slots, c.cache, 16)
    clean, lse0 = c.run(return_lse=True)
    q = c.q.clone()
    q[0, 1, 5] = float("inf")
    q[-1, 2, 5] = float("inf")
    o, lse = c.run(q=q, return_lse=True)
    for at in ((0, 1), (q.shape[0] - 1, 2)):
        assert o[at].isnan().all() and torch.isneginf(lse[at])
        o[at], lse[at] = clean[at], lse0[at]
    assert torch.equal(o, clean) and torch.equal(lse, lse0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40, 200])
def test_the_longest_lengths(new, dtype):
    """2^31 - 16 keys, the longest that a block table of 16-token pages stands for: the last keys within a window as in a
    short request, and (single tokens) all of them, on one page again and again."""
    pages = 2 ** 27 - 1
    c = Case([496], [new], 1, 1, 64, 16, dtype, seed=51)  # ends as the long one does within a tile
    table = torch.zeros((1, pages), dtype=torch.int32, device="cuda")
    table[0, -31:] = c.args[1][0, :31]
    table[0, :-31] = c.args[1][0, 0]
    st, cu, q = status_word(), c.args[3], c.q.cuda()
    o, lse = kda.cache4_attention(q, c.cache, table, dev([pages * 16]), cu, 16, window=100, return_lse=True, status=st)
    want, want_lse = c.run(window=100, return_lse=True)
    assert st.item() == 0 and near(o, want) and (lse - want_lse).abs().max() <= 2.0 ** -16 * (1 + want_lse.abs().max())
    if new == 1:
        o, lse = kda.cache4_attention(0 * q, c.cache, table, dev([pages * 16]), cu, 16, return_lse=True)
        _, v = kda.cache4_read(c.cache, c.args[1][0, 0] * 16 + torch.arange(16, device="cuda").int(), 16, 64, torch.float32)
        # equal weights: the mean over the page that all but 31 of 2^27 entries name
        assert (lse - np.log(pages * 16.0)).abs().max() <= 2.0 ** -16
        assert ((o[0] - v.mean(0)).abs() <= 2.0 ** -8 * v.abs().mean(0) + 2.0 ** -16).all()


def shares(c, rows, tile, lead, workers, window):
    """(items that one worker holds whole, those of one key tile that follow another of its items with key tiles), as the
    kernels divide the work: items request by request, head by head, row tiles from both ends in turn; every worker
    takes an equal, contiguous range of their units."""
    H, G = c.cache.shape[1], c.q.shape[1] // c.cache.shape[1]
    items = []  # units, key tiles
    for L, n in zip(c.lengths, c.new):
        count, t = -(-n * G // rows), -(-L // tile)
        if window:
            t = min(t, (window + (rows - 1) // G + 1) // tile + 2)
        for _, i in itertools.product(range(H), range(count)):
            rt = count - 1 - i // 2 if i % 2 else i // 2
            first, last = L - n + rt * rows // G, L - n + (min(n * G, (rt + 1) * rows) - 1) // G
            low = max(0, first - window + 1) // tile if window else 0
            items.append((max(t, 1) + lead, last // tile + 1 - low if last >= 0 else 0))
    share = max(1, -(-sum(u for u, _ in items) // workers))
    at, whole, short, tiles_before = 0, 0, 0, {}
    for units, tiles in items:
        a, b = at // share, (at + units - 1) // share
        whole += a == b
        short += a == b and tiles == 1 and a in tiles_before
        if tiles:
            tiles_before[b] = True
        at += units
    return whole, short


KINDS = ["few8", "few16", "f32", "many128", "many256"]  # by the rows of a tile; f32 has 8


def crowd(kind, d, window=0, **kw):
    """A batch of so many requests that workers go from item to item, and what check() takes: rows come out of the
    attention kernels themselves, contexts of one tile, of odd tiles and of none follow one another."""
    R, H, G, most = dict(few8=(1500, 3, 2, 1), few16=(1000, 2, 8, 2), f32=(400, 2, 3, 9), many128=(110, 4, 3, 40),
                         many256=(70, 3, 2, 120))[kind]
    r = np.random.default_rng(R + d + window)
    lengths = np.where(r.random(R) < 0.4, r.integers(0, 70, R), r.integers(1, 300, R)).tolist()
    least = {"many128": 6, "many256": 70}.get(kind, 1)  # more than 16 rows, more than 128 rows
    new = r.integers(least, most + 1, R).tolist()
    c = Case(lengths, new, H * G, H, d, 16, "f32" if kind == "f32" else "bf16", seed=R + d, ks=[0.5, 4.0, 1.0, 2.0][:H],
             vs=[1.0, 2.0 ** -6, 3.0, 1.0][:H], **kw)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows, tile, lead, workers = {"few8": (8, 64, 2, 12 * sms), "few16": (16, 64, 2, 12 * sms), "f32": (8, 64, 2, 12 * sms),
                                 "many128": (128, 128, 5, sms), "many256": (256, 128, 5, sms)}[kind]
    whole, short = shares(c, rows, tile, lead, workers, window)
    assert whole >= R // 2 and short >= R // 8
    return c, dict(window=window, max_new=most)


@pytest.mark.parametrize("window", [0, 50])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", KINDS)
def test_workers_that_hold_whole_items(kind, d, window):
    c, how = crowd(kind, d, window)
    o, lse = c.check(**how)
    for _ in range(3):
        again = c.run(return_lse=True, **how)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def positions(c):
    """Of every query row."""
    return torch.cat([torch.arange(L - n, L) for L, n in zip(c.lengths, c.new)])


@pytest.mark.parametrize("kind", KINDS)
def test_whole_items_whose_scores_are_minus_infinity(kind):
    """As test_scores_of_minus_infinity_alone_are_not_an_empty_row, in rows that no join makes; their neighbours keep
    their bits."""
    c, how = crowd(kind, 64)
    c.k[:, :, 5] = -3.0
    kda.cache4_append(c.k.bfloat16().cuda(), c.v.bfloat16().cuda(), c.slots, c.cache, 16, k_scale=c.ks, v_scale=c.vs)
    clean, lse0 = c.run(return_lse=True, **how)
    q = c.q.clone()
    q[::7, 1, 5] = float("inf")
    o, lse = c.run(q=q, return_lse=True, **how)
    seen = (positions(c)[::7] >= 0).cuda()
    assert o[::7, 1][seen].isnan().all() and (o[::7, 1][~seen] == 0).all() and torch.isneginf(lse[::7, 1]).all()
    o[::7, 1], lse[::7, 1] = clean[::7, 1], lse0[::7, 1]
    assert torch.equal(o, clean) and torch.equal(lse, lse0)


@pytest.mark.parametrize("power", [22, 30])
@pytest.mark.parametrize("kind", KINDS)
def test_whole_items_of_scores_far_apart(kind, power):
    """Every row is finite and within its values' range at scores of 2^power, and a query that sees one key gets its value
    (bounds as in test_scores_far_apart)."""
    c, how = crowd(kind, 128, gain=2.0 ** power)
    o, lse = c.run(return_lse=True, **how)
    o, lse, at = to64(o), to64(lse), positions(c).numpy()
    rel = 2.0 ** -19 if kind == "f32" else 2.0 ** -8 + 2.0 ** -11
    assert np.isfinite(o).all() and np.isfinite(lse[at >= 0]).all() and np.isneginf(lse[at < 0]).all()
    _, values = ref.decode(c.cache.cpu().numpy(), c.d)
    values, G, ones = values * to64(c.vs)[:, None, None], c.q.shape[1] // c.cache.shape[1], 0
    for r, (n, L) in enumerate(zip(c.new, c.lengths)):
        v = values[c.table[r, :-(-L // 16)]].swapaxes(0, 1).reshape(values.shape[1], -1, c.d)[:, :L]
        largest = np.maximum.accumulate(np.abs(v), axis=1)
        for i in range(n):
            row, pos = c.cu[r] + i, L - n + i
            if pos < 0:
                assert np.all(o[row] == 0)
                continue
            assert np.all(np.abs(o[row]) <= (1 + rel) * np.repeat(largest[:, pos], G, axis=0))
            if pos == 0:
                ones += 1
                only = np.repeat(v[:, 0], G, axis=0)
                assert np.all(np.abs(o[row] - only) <= rel * np.abs(only))
    assert ones > 0


@pytest.mark.parametrize("lengths,new", [([900, 300], [40, 25]), ([900, 300], [200, 30]), ([900, 300, 77], [1, 40, 2]),
                                         ([900, 4000, 77], [1, 200, 1])])
def test_graphs_of_the_many_row_kernel_and_of_both(lengths, new):
    """Replays of the tcgen05 kernel with its join, and of both kernels with theirs, give the call's bits; the inputs change
    between replays."""
    c = Case(lengths, new, 8, 2, 128, 64, seed=61)
    q, side = c.q.cuda(), torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ws = torch.empty(kda.cache4_attention_workspace_size(len(new), sum(new), 8, 2, 128), dtype=torch.uint8, device="cuda")
    call = lambda: kda.cache4_attention(q, *c.args, max_new=max(new), out=out, lse=lse, return_lse=True, workspace=ws)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    side.synchronize()
    for i in range(3):
        q.copy_(torch.roll(c.q, i, 1))
        out.zero_()
        lse.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        want = c.run(q=torch.roll(c.q, i, 1), max_new=max(new), return_lse=True)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_quotients_past_fp32_saturate():
    """Finite rows whose quotient by the head's scale overflows hold the largest value with their sign and mark nothing; a
    scale that is NaN marks its head's tokens."""
    T, H, d, page = 3, 2, 64, 16
    k = torch.ones(T, H, d)
    k[1, 0] = -1e30
    k[1, 0, 20:30] = 1e3
    v, scale = torch.randn(T, H, d), torch.tensor([2.0 ** -40, 1.0])
    cache, st = kda.cache4_alloc(1, H, page, d), status_word()
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    how = dict(k_scale=scale.cuda(), status=st)
    kda.cache4_append(k.cuda(), v.cuda(), slots, cache, page, **how)
    ko, vo = kda.cache4_read(cache, slots, page, d, dtype=torch.float32, **how)
    assert st.item() == 0
    want = np.float32(2688) * np.sign(k[:, 0].numpy()) * np.float32(2.0 ** -40)
    assert np.array_equal(to64(ko)[:, 0], want.astype(np.float64)) and np.array_equal(to64(ko)[:, 1], ref.held(k.numpy())[:, 1])
    assert np.array_equal(to64(vo), ref.held(v.numpy()))
    how["k_scale"] = torch.tensor([1.0, float("nan")], device="cuda")
    kda.cache4_append(k.cuda(), v.cuda(), slots, cache, page, **how)
    _, vo = kda.cache4_read(cache, slots, page, d, dtype=torch.float32)
    assert st.item() == kda.STATUS_NOT_FINITE and vo[:, 1].isnan().all() and not vo[:, 0].isnan().any()
