"""Workspaces of exactly the queried size, in the middle of larger buffers: the calls write nothing around them, and give
what they give with a workspace of their own."""
import pytest
import torch

import kda_gated_delta_02_gb300 as kda

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BAND = 1 << 20


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _check(need, call, name):
    """call(workspace) with `need` bytes between two bands of 0xa5."""
    assert need > 0, name
    buf = torch.full((BAND + need + BAND,), 0xa5, dtype=torch.uint8, device="cuda")
    ws = buf[BAND:BAND + need]
    got = [t for t in call(ws) if t is not None]
    assert (buf[:BAND] == 0xa5).all() and (buf[BAND + need:] == 0xa5).all(), name
    assert (ws != 0xa5).any(), name  # it was this one that the call used
    for p, q in zip(got, [t for t in call(None) if t is not None], strict=True):
        assert torch.equal(p, q), name


@pytest.mark.parametrize("dtype", DTYPES)
def test_norm(dtype):
    lib, r = kda.load_library(), _gen(1)
    for rows, d, off in ((1, 1, 0), (3, 64, 0), (5000, 128, 0), (5000, 128, 1), (40, 1000, 0), (700, 5120, 0), (700, 5120, 3),
                         (300, 16384, 0), (300, 16383, 0)):
        x, dy = (r(rows, d + off).to(DTYPES[dtype])[:, off:] for _ in range(2))
        w = r(d)
        need = lib.kda_norm_bwd_workspace_size(rows, d, kda.DTYPE_BF16 if dtype == "bf16" else kda.DTYPE_F32)
        _check(need, lambda ws: kda.norm_bwd(x, dy, w, want_dbias=True, workspace=ws), (rows, d, off))


@pytest.mark.parametrize("dtype", DTYPES)
def test_conv(dtype):
    lib, r = kda.load_library(), _gen(2)
    for lens, C, W, off in (([1], 1, 1, 0), ([3, 0, 5], 5, 4, 0), ([300, 7, 129], 1031, 3, 0), ([2000, 77], 520, 4, 0),
                            ([2000, 77], 520, 4, 1), ([900] * 3, 8192, 2, 0)):
        T, cu, w, b = sum(lens), _cu(lens), r(C, W), r(C)
        x, dy = (r(T, C + off).to(DTYPES[dtype])[:, off:] for _ in range(2))
        need = lib.kda_conv_bwd_workspace_size(T, C, W)
        _check(need, lambda ws: kda.conv_bwd(x, w, cu, dy, bias=b, workspace=ws), (lens, C, W, off))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lens,D,G,S,off", [([700, 0, 5, 400, 130], 48, 1, 16, 0), ([700, 0, 5, 400, 130], 47, 1, 8, 1), ([3000], 40, 2, 64, 0),
                                            ([5, 0, 300], 129, 3, 32, 0), ([1, 2, 3] * 20 + [2600], 2048, 1, 16, 0), ([17, 3], 33, 3, 16, 1),
                                            ([1], 1, 1, 8, 0)])
def test_scan(lens, D, G, S, off, dtype):
    lib, r, N, T, cu = kda.load_library(), _gen(3), len(lens), sum(lens), _cu(lens)
    x, dt, z, dy = (r(T, D + off).to(DTYPES[dtype])[:, off:] for _ in range(4))
    B, C = (r(T, G, S).to(DTYPES[dtype]) for _ in range(2))
    args = (x, dt, -torch.exp(r(D, S)), B, C, cu)
    kw = dict(D=r(D), z=z, dt_bias=r(D) - 3, initial_state=r(N, D, S))
    # (`saved` has places that no state belongs to)
    saved, dfinal = torch.zeros(lib.kda_scan_saved_size(N, T, D, S) // 4, device="cuda"), r(N, D, S)
    if need := lib.kda_scan_workspace_size(N, T, D, G, S):
        _check(need, lambda ws: kda.scan_fwd(*args, save=True, saved=saved.clone(), workspace=ws, **kw), "forward")
    else:
        assert T < 256
    kda.scan_fwd(*args, save=True, saved=saved, **kw)
    _check(lib.kda_scan_bwd_workspace_size(N, T, D, G, S),
           lambda ws: kda.scan_bwd(*args, dy, saved, dfinal_state=dfinal, workspace=ws, **kw), "backward")


@pytest.mark.parametrize("lens", [[300, 0, 70], [9, 3]])
def test_saved_states(lens):
    """`saved` of exactly the queried size between two bands."""
    lib, r, D, S, N, T = kda.load_library(), _gen(4), 37, 16, len(lens), sum(lens)
    x, dt, B, C = r(T, D), r(T, D), r(T, 1, S), r(T, 1, S)
    n, band = lib.kda_scan_saved_size(N, T, D, S) // 4, 1 << 16
    buf = torch.full((band + n + band,), 7.0, device="cuda")
    kda.scan_fwd(x, dt, -torch.exp(r(D, S)), B, C, _cu(lens), save=True, saved=buf[band:band + n])
    assert (buf[:band] == 7).all() and (buf[band + n:] == 7).all() and (buf[band:band + n] != 7).any()
