"""Norms and rotation of query and key heads through the public entry point, against 64 bits.

Tolerance, of an output made of the pair (y_a, y_b): the sum of squares rounds at 16 + 4 additions
(20 x 2^-24 of it, half of that in its root), root, inverse, mean, and the products with x, the
inverse and the weight add 6 x 2^-24, sine and cosine are off by 2^-23 each, products and sum by
3 x 2^-24: less than 2^-19 (|y_a| + |y_b|) in all.  bf16 outputs round by 2^-8 of themselves."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():   # pragma: no cover - CPU machine
    pytest.skip("needs a GPU", allow_module_level=True)

from heterogeneous_lora_gemm_gb300 import Rotary, mlora  # noqa: E402

TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets_of(rows):
    return i32(np.concatenate([[0], np.cumsum(rows)]).astype(np.int32))


def plain(x, pos, freq, interleaved, weight, eps):
    """(outputs, |y_a| + |y_b|) in 64 bits; pos [T]."""
    x = x.double().cpu().numpy()
    if weight is not None:
        with np.errstate(all="ignore"):
            size = np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
            x = np.where(size > 0, x / np.where(size > 0, size, 1), 0) * weight.double().cpu().numpy()
    R = 2 * len(freq)
    a, b = (np.arange(0, R, 2), np.arange(1, R, 2)) if interleaved else (np.arange(R // 2), np.arange(R // 2, R))
    angle = pos[:, None, None].astype(np.longdouble) * np.asarray(freq, np.longdouble)
    c, s = np.cos(angle).astype(np.float64), np.sin(angle).astype(np.float64)
    y, size = x.copy(), np.abs(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    y[pos < 0] = 0.0
    return y, size


def check(rows, lengths, heads, D, R, dtype, interleaved=False, norm=(True, True), base=10000.0, eps=1e-6, size=1.0,
          in_place=False, freq=None, seed=0, max_new=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, Hq, H = sum(rows), *heads
    freq = [base ** (-2.0 * i / R) for i in range(R // 2)] if freq is None else freq
    wide = (torch.randn((T, Hq + 2 * H, D), device="cuda", generator=g) * size).to(TDT[dtype])
    before = wide.clone()
    Q, K = wide[:, :Hq], wide[:, Hq:Hq + H]
    weights = [torch.randn(D, device="cuda", generator=g) + 1 if n else None for n in norm]
    outs = [Q, K] if in_place else [torch.full((T, h + 1, D), 5.0, dtype=TDT[dtype], device="cuda")[:, :h] for h in (Hq, H)]
    r = Rotary(D, freq=freq, interleaved=interleaved)
    off = None if set(rows) == {1} else offsets_of(rows)
    r.apply(Q, K, i32(lengths), offsets=off, max_new=max(rows) if max_new is None else max_new, q_weight=weights[0],
            k_weight=weights[1], eps=eps, q_out=None if in_place else outs[0], k_out=None if in_place else outs[1])
    pos = np.concatenate([np.arange(n - k, n) for k, n in zip(rows, lengths)])
    for x, out, w in ((before[:, :Hq], outs[0], weights[0]), (before[:, Hq:Hq + H], outs[1], weights[1])):
        want, scale = plain(x, pos, freq, interleaved, w, eps)
        got = out.double().cpu().numpy()
        tol = 2.0 ** -19 * scale + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0.0) + 1e-37
        bad = ~(np.abs(got - want) <= tol)
        assert not bad.any(), f"{bad.sum()} of {bad.size} off, worst {np.abs(got - want)[bad].max()}, first {np.argwhere(bad)[0]}"
        if not in_place:
            assert torch.all(out._base[:, -1] == 5.0)
    assert torch.equal(wide[:, Hq + H:], before[:, Hq + H:])
    assert r.status() == mlora.MLORA_OK
    return outs


CASES = [
    # rows, lengths, (q heads, kv heads), D, R, interleaved
    ([1], [1], (1, 1), 16, 16, False),
    ([1, 1, 1], [700, 1, 0], (32, 8), 128, 128, False),
    ([1] * 5, [9, 100, 2000, 131072, 7], (3, 5), 64, 64, True),
    ([7, 0, 1, 40], [7, 3, 900, 65], (10, 5), 80, 32, True),
    ([7, 0, 1, 40], [7, 3, 900, 65], (10, 5), 80, 80, False),
    ([3, 5], [2, 5], (4, 2), 96, 48, False),                  # rows at negative positions
    ([1], [2 ** 30], (2, 1), 256, 256, False),                # the farthest position
    ([300, 20], [300, 70000], (6, 1), 256, 16, True),
    ([33], [40], (7, 7), 32, 16, False),
    ([130], [130], (71, 1), 112, 112, False),
    ([1200], [1500], (24, 8), 48, 48, True),
    ([50], [60], (9, 3), 128, 0, False),                      # norms alone
    ([6] * 70, list(range(6, 76)), (2, 2), 64, 64, False),    # more sequences than a warp looks at once
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,lengths,heads,D,R,interleaved", CASES)
def test_matches_64_bits(rows, lengths, heads, D, R, interleaved, dtype):
    a = check(rows, lengths, heads, D, R, dtype, interleaved)
    b = check(rows, lengths, heads, D, R, dtype, interleaved, in_place=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("norm", [(False, False), (True, False), (False, True)])
def test_norms_are_optional(norm, dtype):
    check([5, 1], [5, 900], (8, 2), 128, 128, dtype, norm=norm)


@pytest.mark.parametrize("size,eps", [(1e-18, 1e-6), (1e-18, 0.0), (1e-30, 0.0), (1e18, 1e-6), (1e30, 1e-6), (1e-30, 1e-30), (1e4, 1e3)])
def test_sizes_of_rows_and_eps(size, eps):
    check([5, 1], [5, 900], (3, 2), 80, 80, "f32", size=size, eps=eps)


def test_many_sequences():
    """Empty ones among them; 65535 of them."""
    rng = np.random.default_rng(2)
    rows = rng.integers(0, 3, 3000).tolist()
    check(rows, [int(n + 7) for n in rng.integers(0, 5000, 3000)], (2, 1), 32, 32, "f32", max_new=4)
    check([1] * 65535, rng.integers(1, 100000, 65535).tolist(), (1, 1), 16, 16, "bf16", norm=(False, False))


def test_frequencies_of_any_sign_and_size():
    check([40], [100000], (2, 1), 32, 32, "f32", freq=[-1.0, 3.0, -0.001, 1000.0, 0.0, 2 * np.pi, -1024.0, np.pi / 2,
                                                       1e-9, 0.5, -2.5, 100.0, 7.0, 1e-300, 6.28, 1024.0], norm=(False, False))


def test_a_head_of_zeros_and_values_that_are_no_numbers():
    x = torch.zeros((2, 2, 64), device="cuda")
    x[1, 0, 3] = float("nan")
    x[1, 1] = 1.0
    w = torch.ones(64, device="cuda")
    r = Rotary(64)
    out = torch.full_like(x, 9.0)
    r.apply(x, x.clone(), i32([5, 6]), q_weight=w, eps=0.0, q_out=out)
    assert not out[0].any() and torch.isnan(out[1, 0]).all() and torch.isfinite(out[1, 1]).all()


def test_rows_of_no_sequence_are_left_alone():
    """Before the first range and behind the last; bad ranges; more rows than max_new."""
    x = torch.randn((9, 2, 64), device="cuda")
    r = Rotary(64)

    def run(offsets, lengths, max_new):
        q, k = x.clone(), x.clone()
        r.apply(q, k, i32(lengths), offsets=i32(offsets), max_new=max_new)
        assert torch.equal(q, k)
        return (q != x).any(-1).any(-1).cpu().tolist(), r.status()

    ok, bad = mlora.MLORA_OK, mlora.MLORA_ERR_DEVICE_STEP
    assert run([2, 4, 7], [100, 50], 3) == ([False] * 2 + [True] * 5 + [False] * 2, ok)
    assert run([0, 4, 12], [100, 50], 8) == ([True] * 4 + [False] * 5, bad)          # past T
    assert run([0, 4, 9], [100, 50], 3) == ([True] * 3 + [False] + [True] * 3 + [False] * 2, bad)
    assert run([0, 9, 9], [100, -4], 9) == ([True] * 9, bad)                         # a length below 0, of no row
    assert run([0, 9], [2 ** 31 - 1], 9)[1] == bad                                    # taken as 2^30
    assert run([5, 2], [100], 9) == ([False] * 9, bad)
    assert r.status() == ok                                                           # read and cleared


def test_streams_and_graphs():
    x = torch.randn((50, 3, 128), device="cuda").bfloat16()
    w = torch.randn(128, device="cuda")
    r = Rotary(128)
    lengths, off = i32([30, 90]), offsets_of([20, 30])
    want = [torch.empty_like(x) for _ in range(2)]
    step = dict(offsets=off, max_new=30, q_weight=w, k_weight=w)
    r.apply(x, x, lengths, **step, q_out=want[0], k_out=want[1])
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), [torch.zeros_like(x) for _ in range(2)]
    r.apply(x, x, lengths, **step, q_out=got[0], k_out=got[1], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.apply(x, x, lengths, **step, q_out=got[0], k_out=got[1])
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert r.status(side) == mlora.MLORA_OK


def test_rows_past_32_bit_offsets():
    """Queries of 2^32 elements and more, of which the last rows are looked at."""
    T, Hq, D = 2 ** 19 + 5, 64, 128
    q = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    q[-5:] = torch.randn((5, Hq, D), device="cuda")
    k = torch.empty((T, 1, D), dtype=torch.bfloat16, device="cuda")
    k[-5:] = torch.randn((5, 1, D), device="cuda")
    before = q[-5:].clone()
    r = Rotary(D)
    r.apply(q, k, i32([T + 3]), offsets=offsets_of([T]), max_new=T)
    want, scale = plain(before, np.arange(T - 2, T + 3), [10000.0 ** (-2.0 * i / D) for i in range(D // 2)], False, None, 0)
    got = q[-5:].double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -19 * scale + 2.0 ** -8 * np.abs(want)).all()
    assert r.status() == mlora.MLORA_OK


def test_refusals():
    x = torch.zeros((2, 2, 64), device="cuda")
    r, n = Rotary(64), i32([3, 4])
    for bad in (lambda: r.apply(x, x.bfloat16(), n), lambda: r.apply(x.half(), x.half(), n), lambda: r.apply(x[..., :32], x, n),
                lambda: r.apply(x, x[:1], n), lambda: r.apply(x, x, n.long()), lambda: r.apply(x, x, n.cpu()),
                lambda: r.apply(x, x, n, offsets=n), lambda: r.apply(x.cpu(), x.cpu(), n),
                lambda: r.apply(x, x, n, q_out=x.bfloat16()), lambda: r.apply(x, x, n, k_out=x[:1]),
                lambda: r.apply(x, x, n, q_weight=x[0]), lambda: r.apply(x, x, n, k_weight=torch.ones(64, dtype=torch.bfloat16, device="cuda")),
                lambda: r.apply(x, x, n, q_weight=torch.ones(64)),
                lambda: r.apply(x.transpose(1, 2).contiguous().transpose(1, 2), x, n), lambda: Rotary(64, device="cpu"),
                lambda: Rotary(64, rotary_dim=32, freq=[1.0])):
        with pytest.raises(ValueError):
            bad()
    odd = torch.zeros((2, 130), device="cuda")
    for bad in (lambda: r.apply(x, x, i32([3])), lambda: r.apply(x, x, n, max_new=-1), lambda: r.apply(x, x, n, eps=-1.0),
                lambda: r.apply(x, x, n, eps=float("nan")), lambda: r.apply(x, x, n, q_weight=torch.ones(68, device="cuda")[1:65]), lambda: r.apply(odd[:, 2:].unflatten(1, (2, 64)), x, n),
                lambda: Rotary(64, freq=[float("inf")] * 32)):
        with pytest.raises(mlora.MloraError) as e:
            bad()
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
    none = torch.zeros((0, 2, 64), device="cuda")
    r.apply(none, none, n[:0])
    r.apply(none, none, n[:1], offsets=i32([0, 0]), max_new=3)
    assert r.status() == mlora.MLORA_OK


def test_outputs_that_overlap_are_refused():
    x, k, n = torch.ones((2, 2, 64), device="cuda"), torch.ones((2, 1, 64), device="cuda"), i32([3, 4])
    r = Rotary(64)
    for q_out, k_out in ((x[:1].expand(2, 2, 64), k), (x[:, :1].expand(2, 2, 64), k), (x, k[:1].expand(2, 1, 64)),
                         (x.view(-1).as_strided((2, 2, 64), (128, 32, 1)), k), (x, x[:, :1])):
        with pytest.raises(mlora.MloraError) as e:
            r.apply(x.clone(), k.clone(), n, q_out=q_out, k_out=k_out)
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
    assert torch.all(x == 1) and torch.all(k == 1) and r.status() == mlora.MLORA_OK
    one = torch.ones((1, 64), device="cuda")   # a single row or head has no stride
    r.apply(x[:1, :1].expand(1, 1, 64), one.as_strided((1, 1, 64), (0, 0, 1)), i32([1]))
    assert torch.all(one == 1)   # position 0


@pytest.mark.parametrize("T,heads,row,head", [(2, 2, 1, 1), (2, 32, 1, 1), (3, 6, 5, 2), (11, 4, 3, 10), (2, 5, 8, 2), (40, 33, 2, 64),
                                              (2, 2, 1.25, 1), (2, 2, 1, 1.25), (9, 9, 1.25, 9)])
def test_outputs_whose_rows_lie_among_their_heads_are_refused(T, heads, row, head):
    """Strides of a head and more, in heads: two heads of unequal rows share elements."""
    x, k = torch.ones((T, heads, 64), device="cuda"), torch.ones((T, 1, 64), device="cuda")
    r, n = Rotary(64), i32([T])
    row, head = int(row * 64), int(head * 64)
    out = torch.full(((T - 1) * row + (heads - 1) * head + 64,), 7.0, device="cuda")
    mine = out.as_strided((T, heads, 64), (row, head, 1))
    for kw, q, kk in ((dict(q_out=mine), x, k), (dict(k_out=mine), k, x)):
        with pytest.raises(mlora.MloraError) as e:
            r.apply(q.clone(), kk.clone(), n, offsets=i32([0, T]), max_new=T, **kw)
        assert e.value.status == mlora.MLORA_ERR_INVALID_ARG
    assert torch.all(out == 7.0) and r.status() == mlora.MLORA_OK


@pytest.mark.parametrize("T,heads,row,head", [(2, 4, 5, 2), (3, 3, 1, 3), (5, 4, 4, 1), (2, 2, 3, 2), (3, 2, 2, 7), (2, 3, 1.25, 2.5)])
def test_outputs_whose_rows_lie_among_their_heads_without_overlap(T, heads, row, head):
    row, head = int(row * 64), int(head * 64)
    x, k = torch.randn((T, heads, 64), device="cuda"), torch.randn((T, 1, 64), device="cuda")
    r, n = Rotary(64), i32([T + 5])
    out = torch.full(((T - 1) * row + (heads - 1) * head + 64,), 7.0, device="cuda")
    mine = out.as_strided((T, heads, 64), (row, head, 1))
    want, other = torch.empty_like(x), torch.empty_like(k)
    step = dict(offsets=i32([0, T]), max_new=T, k_out=other)
    r.apply(x, k, n, q_out=want, **step)
    r.apply(x, k, n, q_out=mine, **step)
    assert torch.equal(mine, want)
    mine.fill_(7.0)
    assert torch.all(out == 7.0)      # (what lies between was left alone)


def test_broadcast_inputs():
    """One row for all positions, one head for all heads."""
    x, k = torch.randn((1, 1, 64), device="cuda"), torch.randn((5, 1, 64), device="cuda")
    out = torch.empty((5, 3, 64), device="cuda")
    r = Rotary(64)
    r.apply(x.expand(5, 3, 64), k, i32([9]), offsets=i32([0, 5]), max_new=5, q_out=out)
    want, size = plain(x.expand(5, 3, 64), np.arange(4, 9), [10000.0 ** (-2.0 * i / 64) for i in range(32)], False, None, 0.0)
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -19 * size)
    assert r.status() == mlora.MLORA_OK
