"""Refusals of the 4-bit cache calls (binding and C ABI, no GPU) and the CPU reference's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import cache4_ref as ref
import kda_gated_delta_02_gb300 as kda


def _attn(T=5, Hq=4, H=2, d=64, page=16, R=2, B=3, P=7, dtype=torch.bfloat16):
    return dict(q=torch.zeros(T, Hq, d, dtype=dtype), cache=torch.zeros(P, H, page * 9 * d // 8, dtype=torch.uint8),
                table=torch.zeros(R, B, dtype=torch.int32), seq=torch.zeros(R, dtype=torch.int32),
                cu=torch.zeros(R + 1, dtype=torch.int32), page=page)


def _call(x, **kw):
    return kda.cache4_attention(x["q"], x["cache"], x["table"], x["seq"], x["cu"], x["page"], **kw)


@pytest.mark.parametrize("key,bad,msg", [
    ("q", lambda x: x["q"].half(), "unsupported input dtype"),
    ("q", lambda x: x["q"][:, :3], "multiple of the cache's"),
    ("q", lambda x: x["q"][0], "q must be"),
    ("cache", lambda x: x["cache"].int(), "cache must be uint8"),
    ("cache", lambda x: x["cache"][:, :, 1:], "cache must have shape"),
    ("page", lambda x: 32, "cache must have shape"),
    ("table", lambda x: x["table"].long(), "block_table must be"),
    ("seq", lambda x: x["seq"][:1], "seq_len must have shape"),
    ("cu", lambda x: x["cu"][:-1], "cu_seqlens must have shape"),
    ("cu", lambda x: x["cu"].float(), "cu_seqlens must be"),
])
def test_attention_rejects(key, bad, msg):
    x = _attn()
    x[key] = bad(x)
    with pytest.raises(kda.KDAError, match=msg):
        _call(x)


def test_attention_rejects_outputs_scales_and_host_tensors():
    x = _attn()
    with pytest.raises(kda.KDAError, match="out must be"):
        _call(x, out=torch.zeros(5, 4, 64))
    with pytest.raises(kda.KDAError, match="lse must have shape"):
        _call(x, lse=torch.zeros(4, 5))
    with pytest.raises(kda.KDAError, match="k_scale must have shape"):
        _call(x, k_scale=torch.ones(4))
    with pytest.raises(kda.KDAError, match="CUDA tensors"):
        _call(x)


def test_rows_reject():
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    cache, slots = torch.zeros(3, 2, 16 * 72, dtype=torch.uint8), torch.zeros(5, dtype=torch.int32)
    with pytest.raises(kda.KDAError, match="v must be"):
        kda.cache4_append(k, k.float(), slots, cache, 16)
    with pytest.raises(kda.KDAError, match="k must have shape"):
        kda.cache4_append(k[:, :1], k, slots, cache, 16)
    with pytest.raises(kda.KDAError, match="slot_map must be"):
        kda.cache4_append(k, k, slots.long(), cache, 16)
    with pytest.raises(kda.KDAError, match="slot_map must have shape"):
        kda.cache4_append(k, k, slots[:4], cache, 16)
    with pytest.raises(kda.KDAError, match="slots must"):
        kda.cache4_read(cache, slots[None], 16, 64)
    with pytest.raises(kda.KDAError, match="CUDA tensors"):
        kda.cache4_append(k, k, slots, cache, 16)


def test_plan_rejects():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    good = [i(3), i(3), i(3), i(3, 4), i(9), i(1)]
    for at, bad, msg in ((0, i(2), "context_len must have shape"), (1, i(3).long(), "new_len must be"), (2, i(4), "page_count must"),
                         (3, i(3, 4).float(), "block_table must be"), (4, i(9).long(), "free_pages must be"),
                         (5, i(2), "free_count must have shape")):
        args = list(good)
        args[at] = bad
        with pytest.raises(kda.KDAError, match=msg):
            kda.page_plan(*args, 16, 5)
    with pytest.raises(kda.KDAError, match="tokens"):
        kda.page_plan(*good, 16, -1)


def test_abi_refuses_before_any_launch():
    lib = kda.load_library()
    buf = ctypes.create_string_buffer(128)
    p = (ctypes.addressof(buf) + 15) & ~15
    ws = lib.kda_cache4_attention_workspace_size(2, 5, 8, 2, 128, 0)
    assert ws > 0 and lib.kda_cache4_attention_workspace_size(2, 5, 8, 2, 96, 0) == 0

    def attn(q=p, cache=p, R=2, T=5, Hq=8, H=2, d=128, P=4, page=64, B=3, new=0, window=0, qs=8 * 128, o=p, dt=0, w=p, wb=ws):
        return lib.kda_cache4_attention(q, cache, p, p, p, R, T, Hq, H, d, P, page, B, new, window, 1.0, qs, None, None, o,
                                        None, dt, w, wb, None, None)

    assert attn(d=96) == -2 and attn(page=48) == -2 and attn(page=512) == -2 and attn(Hq=7) == -2 and attn(P=2 ** 25 + 1) == -2
    assert attn(R=0) == -1 and attn(T=-1) == -1 and attn(window=-1) == -1 and attn(new=-1) == -1 and attn(dt=2) == -1
    assert attn(q=None) == -1 and attn(cache=None) == -1 and attn(qs=8 * 128 - 8) == -1 and attn(P=0) == -1
    assert attn(q=p + 4) == -3 and attn(o=p + 8) == -3 and attn(qs=8 * 128 + 4) == -3
    assert attn(wb=ws - 1) == -4 and attn(w=None) == -4

    def append(k=p, slots=p, T=3, H=2, d=64, P=2, page=16, ks=128, vs=128, dt=0):
        return lib.kda_cache4_append(k, p, slots, p, T, H, d, P, page, ks, vs, None, None, dt, None, None)

    assert append(d=32) == -2 and append(page=8) == -2 and append(T=-1) == -1 and append(k=None) == -1 and append(slots=None) == -1
    assert append(k=p + 2) == -3 and append(ks=120) == -1 and append(vs=132) == -3 and append(dt=1, ks=130) == -3
    assert append(T=0) == 0 and append(T=2 ** 31 - 1, H=3, ks=192, vs=192) == -2 and attn(T=2 ** 31 - 1) == -2

    def read(out=p, n=3, P=2):
        return lib.kda_cache4_read(p, p, n, 2, 64, P, 16, None, None, 0, out, p, None, None)

    assert read(out=None) == -1 and read(n=-1) == -1 and read(P=2 ** 28) == -2 and read(n=0) == 0

    def plan(R=2, B=3, F=4, page=16, T=3, count_out=p + 16, free_out=p + 16, slots=p):
        return lib.kda_page_plan(p, p, p, p, p, p, R, B, F, page, T, p, p, slots, p, count_out, free_out, None, None)

    assert plan(R=0) == -1 and plan(T=-1) == -1 and plan(page=20) == -2 and plan(B=2 ** 27 + 1) == -2 and plan(slots=None) == -1
    assert plan(count_out=p) == -1 and plan(free_out=p) == -1  # in place is not allowed


def test_plan_refuses_outputs_over_inputs():
    """Every output over every input and every other output: from the start, and by one element at either end."""
    lib = kda.load_library()
    R, B, F, T, page = 3, 4, 9, 7, 16
    sizes = dict(context_len=R, new_len=R, page_count=R, block_table=R * B, free_pages=F, free_count=1, cu_seqlens=R + 1,
                 seq_len=R, slot_map=T, positions=T, page_count_out=R, free_count_out=1)
    names = list(sizes)
    buf = ctypes.create_string_buffer(4 * sum(sizes.values()) + 4096)
    at, start = {}, (ctypes.addressof(buf) + 2047) & ~15
    for n in names:  # back to back
        at[n], start = start, start + 4 * sizes[n]
    outputs = names[6:] + ["block_table"]

    def plan(at):
        return lib.kda_page_plan(*(at[n] for n in names[:6]), R, B, F, page, T, *(at[n] for n in names[6:]), None, None)

    for o in outputs:
        for n in names:
            if n == o:
                continue
            for shift in (0, sizes[n] - 1, -(sizes[o] - 1)):
                assert plan({**at, o: at[n] + 4 * shift}) == -1, (o, n, shift)


def test_the_current_stream_without_torchs_internal_function(monkeypatch):
    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(kda, "_raw_stream", None, raising=False)
    assert kda._stream(None) == 0x1234 and kda._stream(Stream) == 0x1234
    monkeypatch.setattr(kda, "_raw_stream", lambda device: 0x100 + device, raising=False)
    assert kda._stream(None) == 0x103


def test_reference_rounding():
    """The reference's nearest() and quantise() on values whose answers are known."""
    assert [ref.E2M1[ref.nearest(np.array(x), ref.E2M1)] for x in (0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 9.0)] == \
        [0.0, 0.5, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 6.0]
    x = np.zeros((1, 16), dtype=np.float32)
    x[0, :4] = [6.0, -3.0, 0.25, 5.0]
    c, s = ref.quantise(x)
    assert ref.E4M3[s[0, 0]] == 1.0 and ref.value(c, s)[0, :4].tolist() == [6.0, -3.0, 0.0, 4.0]
    y = torch.randn(64, 64).numpy()
    t = torch.from_numpy(np.abs(y).reshape(64, 4, 16).max(-1) / np.float32(6)).to(torch.float8_e4m3fn)
    assert np.array_equal(ref.quantise(y)[1], t.view(torch.uint8).numpy())
