"""Low-rank adapters of many requests against float64: types, ranks, odd widths and
pitches, groups from none to many rows, rows without an adapter, updates in place."""
import pytest
import torch

from tests import block_reference as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def A():
    from mixture_experts_ffn_fp32_gb300 import build
    build.build()
    from mixture_experts_ffn_fp32_gb300 import api
    return api


@pytest.fixture(params=["chosen", "few", "many"])
def form(request, monkeypatch):
    """Each form by itself, where a call's operands let it; FP32 has one."""
    if request.param == "chosen":
        monkeypatch.delenv("MOE_ADAPTER_FORM", raising=False)
    else:
        monkeypatch.setenv("MOE_ADAPTER_FORM", request.param)


def make(T, d, N, r, E, dt=torch.bfloat16, out=None, ids=None, pad=0, seed=0, order=True):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*s):
        return torch.randn(*s, generator=g, device="cuda")
    if ids is None:  # some without (E), some adapters without rows
        ids = torch.randint(E + 1, (T,), generator=g, device="cuda")
    ids = torch.as_tensor(ids, device="cuda").long()
    s = {"x": rand(T, d + pad).to(dt)[:, :d], "a": (rand(E, r, d) / d ** 0.5).to(dt), "b": (rand(E, N, r)).to(dt),
         "scale": 0.5 + torch.rand(E, generator=g, device="cuda"), "base": rand(T, N + pad).to(out or dt)[:, :N]}
    s["rows"] = torch.argsort(ids, stable=True).to(torch.int32) if order else None
    n = torch.bincount(ids, minlength=E + 1)[:E]
    s["offsets"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
    return s


def check(got, s, dtype=None):
    val, tol = B.adapter_add(s["base"], s["x"], s["a"], s["b"], s["offsets"], s["rows"], s["scale"], got.dtype,
                             2 if got.dtype != torch.float32 else 3)
    bad = ~((got.double() - val).abs() <= tol * 1.001 + 1e-30)  # a NaN is bad
    assert not bad.any(), (int(bad.sum()), float((got.double() - val).abs()[bad].max()))


# T, d, N, r, E
SIZES = [(1, 64, 64, 16, 1), (1, 4096, 2048, 16, 8), (2, 128, 96, 8, 300), (17, 100, 60, 4, 3), (64, 256, 512, 16, 5),
         (128, 512, 256, 32, 40), (129, 1411, 1003, 12, 7), (200, 768, 520, 64, 2), (300, 2048, 1408, 16, 1),
         (5, 33, 7, 1, 2), (77, 72, 40, 3, 9), (513, 256, 264, 128, 6), (260, 192, 328, 256, 3), (1000, 64, 2000, 24, 1000),
         (33, 8192, 64, 48, 4), (700, 96, 4104, 40, 11), (40, 24, 16, 16, 1024), (2100, 320, 136, 64, 3)]


@pytest.mark.parametrize("dt,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(A, form, size, dt, out):
    s = make(*size, DT[dt], DT[out])
    check(A.adapter_add(**s), s)


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("pad", [1, 4, 8])
def test_pitches(A, form, dt, pad):
    s = make(150, 256, 192, 16, 6, DT[dt], pad=pad)
    check(A.adapter_add(**s), s)
    s = make(150, 257, 193, 16, 6, DT[dt], pad=pad)
    check(A.adapter_add(**s), s)


@pytest.mark.parametrize("per", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 255, 257])
def test_rows_per_adapter(A, form, per):
    """Groups of equal length around every tile's."""
    E = 5
    ids = torch.arange(E).repeat_interleave(per)
    for out in (None, torch.float32):
        s = make(E * per, 256, 320, 16, E, ids=ids, out=out)
        check(A.adapter_add(**s), s)
        s["rows"] = None
        check(A.adapter_add(**s), s)


@pytest.mark.parametrize("T,r", [(1, 16), (64, 16), (900, 64)])
def test_nobody_has_one(A, form, T, r):
    s = make(T, 128, 256, r, 4, ids=torch.full((T,), 4))
    assert torch.equal(A.adapter_add(**s), s["base"])


@pytest.mark.parametrize("T", [3, 300, 3000])
@pytest.mark.parametrize("base", [True, False])
def test_unscaled_and_without_base(A, form, T, base):
    s = make(T, 192, 136, 16, 5)
    s["scale"] = None
    if not base:
        s["base"] = None
    got = A.adapter_add(**s)
    assert got.dtype == torch.bfloat16
    check(got, s)
    if not base:
        none = s["rows"][int(s["offsets"][-1]):].long()
        assert (got[none] == 0).all()


@pytest.mark.parametrize("T,r", [(6, 16), (250, 16), (4000, 64)])
@pytest.mark.parametrize("dt", list(DT))
def test_in_place(A, form, T, r, dt):
    s = make(T, 256, 384, r, 3, DT[dt], pad=8)
    want = A.adapter_add(**s)
    got = A.adapter_add(**s, out=s["base"])
    assert got is s["base"] and torch.equal(got, want)


@pytest.mark.parametrize("T", [40, 2000])
def test_rows_not_named_stay(A, form, T):
    """Bad indices are skipped and flagged; the rows that no position names are not written."""
    s = make(T, 128, 128, 16, 3, ids=torch.arange(T) % 3)
    ws = A.alloc_adapter_workspace(T, 128, 128, 16, 3)
    out = torch.full_like(s["base"], 7.0)
    want = A.adapter_add(**s, ws=ws)
    assert A.workspace_status(ws) == A.MOE_OK
    lost = [int(s["rows"][5]), int(s["rows"][T - 1])]
    s["rows"][5], s["rows"][T - 1] = -3, T + 9
    A.adapter_add(**s, out=out, ws=ws)
    assert A.workspace_status(ws) == A.MOE_ERR_DEVICE_INDEX and A.workspace_status(ws) == A.MOE_OK
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[lost] = False
    assert torch.equal(out[keep], want[keep]) and (out[lost] == 7).all()


@pytest.mark.parametrize("T", [30, 3000])
def test_offsets_out_of_range(A, form, T):
    """Clamped: nothing is read or written outside."""
    s = make(T, 128, 128, 16, 4, ids=torch.arange(T) % 4)
    s["offsets"] = torch.tensor([0, T // 2, T // 2, T + 1000, T + 2000], dtype=torch.int32, device="cuda")
    check(A.adapter_add(**s), s)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T", [50, 3000])
def test_infinite_rows_stay_alone(A, form, T, dt):
    """A row's infinity or NaN reaches that row alone, and an infinity with weights of one sign stays one."""
    s = make(T, 256, 128, 12, 3, DT[dt], ids=torch.arange(T) % 3)
    want = A.adapter_add(**s)
    s["x"][7, 9], s["x"][T - 2, 0] = float("inf"), float("nan")
    got = A.adapter_add(**s)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[7, T - 2]] = False
    assert torch.equal(got[keep], want[keep])
    assert not got[7].isfinite().any() and got[T - 2].isnan().all()
    s["a"].abs_()
    s["b"].abs_().add_(0.1)
    s["x"].abs_()
    assert (A.adapter_add(**s)[7] == float("inf")).all()


@pytest.mark.parametrize("T", [20, 2000])
def test_large_inner_values(A, form, T):
    """FP16 adapters whose inner values leave FP16's range, and some far below their row's largest."""
    s = make(T, 512, 136, 16, 2, torch.float16, torch.float32, ids=torch.arange(T) % 2)
    s["x"] *= 64
    s["a"] *= 64
    s["a"][:, 3] /= 4096
    s["b"] /= 16
    check(A.adapter_add(**s), s)


def test_dispatch_gives_the_groups(A):
    T, E = 513, 6
    ids = torch.randint(E + 1, (T,), generator=torch.Generator().manual_seed(3)).cuda()
    s = make(T, 128, 192, 16, E, ids=ids)
    plan = A.dispatch(A.LayerSpec(T=T, d=128, d_ff=128, E=E + 1, K=1), ids[:, None].int().contiguous(),
                      torch.ones(T, 1, device="cuda"))
    assert torch.equal(plan["offsets"][:E + 1], s["offsets"]) and torch.equal(plan["sorted_token"], s["rows"])
    got = A.adapter_add(s["base"], s["x"], s["a"], s["b"], plan["offsets"][:E + 1], plan["sorted_token"], s["scale"])
    check(got, s)


def test_streams_and_graphs(A, form):
    for T in (60, 3000):
        s = make(T, 256, 512, 16, 9)
        eager = A.adapter_add(**s)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        there = A.adapter_add(**s, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(eager, there)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = A.adapter_add(**s)
        s["x"].neg_()
        # another grouping of the same rows: sizes of groups are read at replay
        s["rows"].copy_(torch.randperm(T, device="cuda"))
        s["offsets"].copy_((torch.arange(10, device="cuda") * (T // 10)).int())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, A.adapter_add(**s))
        check(out, s)


@pytest.mark.parametrize("dt", list(DT))
def test_no_rows(A, dt):
    s = make(0, 64, 96, 16, 3, DT[dt])
    assert A.adapter_add(**s).shape == (0, 96)


@pytest.mark.parametrize("dt", list(DT))
def test_a_workspace_serves_fewer_rows(A, form, dt):
    """One workspace, made for the largest call, for all smaller ones."""
    ws = A.alloc_adapter_workspace(3000, 2048, 96, 16, 4, DT[dt])
    for T in (3000, 1500, 700, 300, 90, 33, 7, 1):
        s = make(T, 2048, 96, 16, 4, DT[dt])
        check(A.adapter_add(**s, ws=ws), s)
    assert A.workspace_status(ws) == A.MOE_OK


def test_large_pitches(A, form):
    """Offsets of rows past 32 bits."""
    T, d, N = 70, 64, 64
    pitch = (1 << 31) // 64
    for T in (70, 1100):
        s = make(T, d, N, 16, 3)
        x = torch.empty(1, dtype=torch.bfloat16, device="cuda").new_empty(pitch * 70 + 64)
        step = pitch * 70 // T // 8 * 8
        s["x"] = torch.as_strided(x, (T, d), (step, 1)).copy_(s["x"])
        check(A.adapter_add(**s), s)
        y = x.new_empty(pitch * 70 + 64)
        s["base"] = torch.as_strided(y, (T, N), (step, 1)).copy_(s["base"])
        want = A.adapter_add(**s)
        assert torch.equal(A.adapter_add(**s, out=s["base"]), want)
        del x, y


def test_two_calls_at_once(A, form):
    """Calls on two streams, each with its own workspace."""
    for T in (100, 2500):
        cases = [make(T, 512, 640, 64, 5, seed=i) for i in range(2)]
        want = [A.adapter_add(**s) for s in cases]
        streams = [torch.cuda.Stream() for _ in cases]
        for st in streams:
            st.wait_stream(torch.cuda.current_stream())
        got = [[], []]
        for _ in range(10):
            for i, (s, st) in enumerate(zip(cases, streams)):
                got[i].append(A.adapter_add(**s, stream=st))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_what_earlier_calls_left(A, form, size, dt):
    """NaNs in shared and tensor memory, in the workspace, between a row's end and its pitch, and in
    rows and adapters that no position joins reach no result."""
    T, d, N, r, E = size
    dtype, nan = DT[dt], float("nan")
    s = make(T, d, N, r, E, dtype, pad=8)
    whole = {k: torch.full((T, n + 8), nan, device="cuda", dtype=dtype) for k, n in (("x", d), ("base", N))}
    for k, n in (("x", d), ("base", N)):
        whole[k][:, :n] = s[k]
        s[k] = whole[k][:, :n]
    dirty = make(2000, 512, 512, min(256, -(-r // 16) * 16), 3, dtype, ids=torch.arange(2000) % 3)
    for k in ("x", "a", "b"):
        dirty[k].fill_(nan)
    ws = A.alloc_adapter_workspace(T, d, N, r, E, dtype)
    ws[256:] = 255
    want = {k: v.clone() if v is not None else None for k, v in s.items()}
    s["x"][s["rows"][int(s["offsets"][E]):].long()] = nan
    empty = (s["offsets"][1:] == s["offsets"][:-1])
    s["a"][empty] = nan
    s["b"][empty] = nan
    s["scale"][empty] = nan
    torch.cuda.synchronize()
    A.adapter_add(**dirty)
    got = A.adapter_add(**s, ws=ws)
    assert A.workspace_status(ws) == A.MOE_OK
    check(got, want)
