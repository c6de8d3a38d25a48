"""The 8-bit operators on the GPU at their limits: moments near the smallest numbers, steps of more than one launch,
products whose sums are split, the 8-bit instruction's own error, and arrays past 2^31 values."""
import numpy as np
import pytest
import torch

import qlora_fine_tuning_quantize_amd as q
from tests import ref8
from tests.helpers import f64, host
from tests.test_gpu_8bit import DEV, DTYPES, Many, assert_product, bits8, matrix

pytestmark = pytest.mark.gpu


# ---- AdamW over many tensors ----

@pytest.mark.parametrize("grad,eps", [("fp32", 1e-8), ("fp32", 1e-15), ("fp32", 1e-30), ("bf16", 1e-30)])
def test_adamw_many_small_second_moments(grad, eps):
    """Gradients whose squares are subnormal in fp32, or vanish, under an eps that does not hide them: parameters stay
    within 2^-21 of their step, which the root of a second moment taken for 0 would make up to 1e10 times as large."""
    print(f"adamw_many small second moments {grad} eps={eps}", flush=True)
    t = Many([5000, 257, 1024, 3], grad, "bf16", 8, 31)
    gen = torch.Generator().manual_seed(32)
    for i, n in enumerate(t.sizes):
        # 1e-13 .. 1e-24: of (1 - beta2) g^2 the normal, the subnormal and what is below the smallest number
        size = 10.0 ** -(13 + 11 * torch.rand(n, generator=gen, dtype=torch.float64))
        t.g[i] = (size * (1 - 2 * torch.randint(0, 2, (n,), generator=gen))).to(DTYPES[grad])
        t.dg[i].copy_(t.g[i])
        for codes, scale in (t.m[i], t.v[i]):
            codes[:], scale[:] = 0, 0
        for x in (t.dm[i].view(torch.uint8), t.dv[i].view(torch.uint8), t.dms[i], t.dvs[i]):
            x.zero_()
    for step in (1, 2, 3):
        q.adamw_step_many(t.plan, lr=1e-3, step=step, eps=eps, seed=5)
        t.step(step, None, 5, lr=1e-3, eps=eps)
        torch.cuda.synchronize()
        t.check(f"step {step}")


def test_adamw_table_is_the_structs():
    """The kernel reads the structs, each tensor's n among them, from device memory: they are the host's, byte for byte."""
    t = Many([5, 0, 300, 1025], "bf16", "fp16", 8, 41)
    assert t.plan._table.dtype == t.plan._structs.dtype and t.plan._table.is_contiguous()
    assert torch.equal(t.plan._table.cpu(), t.plan._structs)
    assert t.plan._structs[:, 7].tolist() == t.sizes
    assert t.plan._structs[:, 0].tolist() == [x.data_ptr() for x in t.dp]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [960, 961, 2000])
def test_adamw_many_launches(bits, count):
    """As many tensors as a launch takes (960), one more, and three launches' worth, some of them empty, at a launch's
    borders too: every tensor is updated once, and 8-bit moments are rounded by the tensor's place among all."""
    print(f"adamw_many launches bits={bits} count={count}", flush=True)
    sizes = [(37 * i) % 611 if i % 5 else 0 for i in range(count)]
    for i, n in ((0, 0), (1, 1300), (63, 2000), (64, 3), (958, 700), (959, 0), (960, 0), (961, 1025), (1918, 5),
                 (1919, 1), (1920, 513)):
        if i < count:
            sizes[i] = n
    sizes[-1] = 300
    t = Many(sizes, "bf16", "bf16", bits, 51)
    for step in (1, 2):
        q.adamw_step_many(t.plan, lr=2e-3, step=step, seed=77)
        t.step(step, None, 77, lr=2e-3)
        torch.cuda.synchronize()
        t.check(f"step {step}")


def test_adamw_many_launches_equal_one_by_one():
    """With 32-bit moments and more tensors than a launch takes: adamw_step on each tensor, bit for bit."""
    t = Many([1 + (64 * i) % 449 for i in range(1100)], "fp32", "bf16", 32, 52)
    one = [[x.clone() for x in xs] for xs in (t.dp, t.dg, t.dm, t.dv, t.copy)]
    q.adamw_step_many(t.plan, lr=1e-3, step=4)
    for p, g, m, v, c in zip(*one):
        q.adamw_step(p, g, m, v, lr=1e-3, step=4, param_bf16=c)
    torch.cuda.synchronize()
    for got, want in zip((t.dp, t.dg, t.dm, t.dv, t.copy), one):
        for x, y in zip(got, want):
            assert torch.equal(x, y)


# ---- products ----

SPLIT = [(300, 130, 5000), (130, 258, 6000), (128, 256, 14336)]


def split_case(M, N, K, dtype):
    """A product whose sums go through the workspace, and its exact factors."""
    assert int(q.lib().ql_fp8_workspace_bytes(M, N, K)) > 0, "the shape is no longer split: take another"
    rng = np.random.default_rng(M + N + K)
    a, av = matrix(M, K, "e5m2", rng.standard_normal((M, K)))
    b, bv = matrix(N, K, "e4m3", rng.standard_normal((N, K)))
    return dict(a=a, b=b, av=av, bv=bv, out=torch.empty(M, N, dtype=DTYPES[dtype], device=DEV),
                ws=q.fp8_matmul_workspace(M, N, K, DEV))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_split_products_on_two_streams(dtype):
    """Products in slices on several streams at once, each with its own workspace, equal the ones run alone."""
    print(f"split products on streams {dtype}", flush=True)
    cases = [split_case(*s, dtype) for s in SPLIT]
    for c in cases:
        c["want"] = q.fp8_matmul(c["a"], c["b"], dtype=DTYPES[dtype])
        assert_product(c["want"], c["av"], c["bv"], dtype)
        c["stream"] = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for c in cases:
            with torch.cuda.stream(c["stream"]):
                q.fp8_matmul(c["a"], c["b"], out=c["out"], ws=c["ws"])
    torch.cuda.synchronize()
    for c in cases:
        assert torch.equal(c["out"], c["want"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_split_products_captured(dtype):
    """Products in slices in two captured graphs that share one workspace, replayed in turn with eager products between
    them and with new operands, equal the eager ones; fp32 ones are added to what is there."""
    print(f"split products captured {dtype}", flush=True)
    cases = [split_case(*s, dtype) for s in SPLIT]
    add = dtype == "fp32"
    ws = max((c["ws"] for c in cases), key=lambda t: t.numel())
    run = lambda c, out, ws: q.fp8_matmul(c["a"], c["b"], out=out, accumulate=add, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in cases:
            c["eager"] = torch.zeros_like(c["out"])
            run(c, c["out"].zero_(), ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for part in (cases[:2], cases[1:]):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for c in part:
                run(c, c["out"], ws)
    for c in cases:
        c["out"].zero_()
        c["eager"].zero_()
    for rep in range(4):
        for g, part in zip(graphs, (cases[:2], cases[1:])):
            for c in part:
                run(c, c["eager"], c["ws"])
            g.replay()
        torch.cuda.synchronize()
        for c in cases:
            assert torch.equal(c["out"], c["eager"]), rep
            if rep == 0 and not add:
                assert_product(c["out"], c["av"], c["bv"], dtype)
        if rep == 1:  # new codes reach the captured products
            for c in cases:
                c["a"].codes.view(torch.uint8).copy_(c["a"].codes.view(torch.uint8).flip(0))


def cut_products(av, bv):
    """What the 8-bit matrix instruction leaves out of a b^T: of each product what is below the bit 2^-13 of the largest
    of its 8 consecutive ones."""
    p = (av[:, None, :] * bv[None, :, :]).reshape(av.shape[0], bv.shape[0], -1, 8)
    largest = np.abs(p).max(3, keepdims=True)
    last = np.ldexp(1.0, np.frexp(np.where(largest > 0, largest, 1.0))[1] - 1 - 13)
    return (p - np.trunc(p / last) * last).sum((2, 3))


@pytest.mark.parametrize("M,N,K,dtype", [(4, 300, 2048, "fp16"), (40, 64, 1024, "bf16"),             # stream
                                         (200, 1000, 2048, "bf16"), (130, 258, 6016, "fp16"),        # 128 x 128, in slices
                                         (1700, 3504, 1024, "bf16"), (3450, 3584, 1024, "fp16")])    # larger tiles
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_matmul_own_error(M, N, K, dtype, fmt):
    """Sums that cancel exactly (normal values against themselves in another order, with the other sign) leave the
    matrix instructions' own error alone, whatever the output's type rounds to.  Its 2-norm over many outputs is at most
    that of the parts cut off, with the accumulator's roundings, and below 2e-5 of the 2-norm of sums that do not cancel.

    The accumulator takes K / 8 sums of 8 and each is off by at most 2^-23 of what is there, with signs of their own: in
    the mean square sqrt(K / 8) 2^-23 of the terms' 2-norm, which bounds that of every partial sum of random signs.  The
    output's rounding is 2^-8 of what is left (bf16).  The parts cut off these sums come to 1.4e-5 to 1.6e-5 in E4M3 and
    1.1e-5 to 1.3e-5 in E5M2 by arithmetic."""
    print(f"matmul own error {M}x{N}x{K} {fmt} {dtype}", flush=True)
    rng = np.random.default_rng(M + N + K)
    order = rng.permutation(K // 2)

    def factor(rows, fmt, flip):
        top = ref8.TOP[fmt]
        codes = ref8.nearest_codes(np.clip(rng.standard_normal((rows, K // 2)) * top / 4.5, -top, top), fmt)
        codes = np.concatenate([codes, codes[:, order] ^ np.uint8(flip)], 1)
        scales = np.full((K // 128, ref8.up(rows, 16)), 122, np.uint8)  # 2^-5
        if fmt == "e5m2":
            scales -= 7
        m = q.FP8Matrix(torch.from_numpy(codes).view(ref8.TYPES[fmt]).to(DEV),
                        torch.from_numpy(scales).to(DEV).view(torch.float8_e8m0fnu), rows, K)
        return m, ref8.dequantize(codes, scales, rows, fmt)
    a, av = factor(M, fmt, 0)
    b, bv = factor(N, "e4m3", 0x80)
    got = q.fp8_matmul(a, b, dtype=DTYPES[dtype])
    torch.cuda.synchronize()
    rows, cols = rng.permutation(M)[:24], rng.permutation(N)[:48]
    av, bv, got = av[rows], bv[cols], f64(host(got))[rows][:, cols]
    norm = lambda v: np.sqrt(np.mean(v ** 2))
    terms = np.sqrt(np.mean((av ** 2) @ (bv ** 2).T))
    assert norm(av @ bv.T) <= 1e-12 * terms
    cut = cut_products(av, bv)
    print(f"  own error {norm(got) / terms:.3e}, cut off {norm(cut) / terms:.3e}", flush=True)
    assert norm(got) <= (1 + 2.0 ** -8) * (norm(cut) + np.sqrt(K / 8) * 2.0 ** -23 * terms)
    assert norm(got) <= 2e-5 * terms


# ---- quantisation ----

def test_quantize_transposed_needs_its_output():
    """A transpose that is asked for is made or refused, never left out."""
    x = torch.ones(20, 300, device=DEV)
    m, mt = q.fp8_quantize(x, transposed=True)
    with pytest.raises(ValueError):
        q.fp8_quantize(x, out=m, transposed=True)
    assert q.fp8_quantize(x, out=m, out_t=mt, transposed=True) == (m, mt)
    assert q.fp8_quantize(x, out_t=mt, transposed=True) == (None, mt)


# ---- past 2^31 values ----

def test_quantize_large():
    """2.15e9 values: codes and scales of the last rows, and of the transpose's last columns."""
    rows, cols = 65541, 32800
    print("quantize large", flush=True)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    for at in range(0, rows, 8192):
        x[at:at + 8192].normal_()
    m, mt = q.fp8_quantize(x, transposed=True)
    alone = q.fp8_quantize(x)
    torch.cuda.synchronize()
    first = rows // 128 * 128 - 128  # the last whole block of rows, and what follows
    tail = f64(host(x[first:]))
    codes, scales, _ = ref8.quantize(tail, 1, "e4m3")
    for got in (m, alone):
        assert np.array_equal(bits8(got.codes[first:]), codes)
        assert np.array_equal(bits8(got.scales)[:, first:rows], scales[:, :rows - first])
    codes, scales, _ = ref8.quantize(tail.T, 1, "e4m3")
    assert np.array_equal(mt.codes.view(torch.uint8)[:, first:].cpu().numpy(), codes)
    assert np.array_equal(bits8(mt.scales)[first // 128:], scales)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_matmul_large(dtype):
    """A matrix of 2.15e9 codes against few rows and as few rows: outputs at its end.  And an output of 2.2e9 values."""
    print(f"matmul large {dtype}", flush=True)
    rows, K = 65541, 32800
    x = torch.empty((rows, K), dtype=torch.bfloat16, device=DEV)
    for at in range(0, rows, 8192):
        x[at:at + 8192].normal_()
    a = q.fp8_quantize(x)
    tail = f64(host(x[-150:]))
    del x
    av = ref8.dequantize(*ref8.quantize(tail, 1, "e4m3")[:2], 150, "e4m3")[:, :K]
    rng = np.random.default_rng(3)
    for n in (5, 70):
        b, bv = matrix(n, K, "e4m3", rng.standard_normal((n, K)))
        assert_product(q.fp8_matmul(a, b, dtype=DTYPES[dtype])[-150:], av, bv, dtype, what=f"many rows x {n}")
        assert_product(q.fp8_matmul(b, a, dtype=DTYPES[dtype])[:, -150:], bv, av, dtype, what=f"{n} x many rows")
    del a
    M, N, K = 47000, 47001, 40
    a, b = (q.fp8_quantize(torch.randn(s, K, device=DEV)) for s in (M, N))
    out = q.fp8_matmul(a, b, dtype=DTYPES[dtype])
    av, bv = (ref8.dequantize(bits8(m.codes[-100:]), bits8(m.scales)[:, s - 100:s], 100, "e4m3")[:, :K]
              for m, s in ((a, M), (b, N)))
    assert_product(out[-100:, -100:], av, bv, dtype, what="many outputs")


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_large(bits):
    """A tensor of 2^31 + 1501 values beside small ones: its end, and the ones after it."""
    print(f"adamw_many large {bits}", flush=True)
    n = 2 ** 31 + 1501
    base = n // 256 * 256 - 4096  # the last values are checked, from a block's border on
    p = [torch.empty(k, device=DEV).normal_() for k in (300, n, 700)]
    g = [torch.empty(k, dtype=torch.bfloat16, device=DEV).normal_() for k in (300, n, 700)]
    plan = q.AdamWTensors.zeros(p, g, bits)
    before = [t[base if t.numel() == n else 0:].cpu().numpy() for t in p]
    q.adamw_step_many(plan, lr=2e-3, step=1, seed=12)
    torch.cuda.synchronize()
    for i, k in enumerate((300, n, 700)):
        at = base if k == n else 0
        gv = f64(host(g[i][at:])).astype(np.float32)
        zero = np.zeros(len(gv), np.float32)
        want, m, v = ref8.adamw(before[i], gv, zero, zero, lr=2e-3, step=1)
        got = p[i][at:].cpu().numpy()
        if bits == 32:
            assert np.array_equal(got, want), i
            assert np.array_equal(plan.exp_avgs[i][at:].cpu().numpy(), m), i
            assert np.array_equal(plan.exp_avg_sqs[i][at:].cpu().numpy(), v), i
            continue
        # the bound of Many.check
        moved = np.abs(want.astype(np.float64) - before[i] * (1 - 2e-3 * 0.01))
        assert np.all(np.abs(got.astype(np.float64) - want) <= 2.0 ** -21 * moved + 4 * 2.0 ** -24 * np.abs(want)), i
        words = np.stack(ref8.philox(np.arange(at // 4, -(-k // 4)), i, 1, 12), 1).reshape(-1)[:k - at].astype(np.int64)
        for codes, scale, x, fmt, r in ((plan.exp_avgs, plan.exp_avg_scales, m, "e4m3", words & 0xFFFF),
                                        (plan.exp_avg_sqs, plan.exp_avg_sq_scales, v, "e5m2", words >> 16)):
            c, s = ref8.store8(x, fmt, r)
            assert np.array_equal(bits8(codes[i][at:]), c), (i, fmt)
            assert np.array_equal(scale[i][at // 256:].cpu().numpy(), s[:-(-len(x) // 256)]), (i, fmt)


# ---- streams and graphs ----

@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_moments_made_here_on_another_stream(bits):
    """A step on another stream, whose object, and with it the moments that zeros() made, is dropped right after the
    call: what takes their memory next neither changes the step nor is written by it."""
    print(f"adamw moments made here {bits}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(61)
    sizes = [70000, 300, 128 * 1024]
    p, g = ([torch.randn(n, generator=gen, device=DEV) for n in sizes] for _ in range(2))
    want = [x.clone() for x in p]
    plain, dropped = q.AdamWTensors.zeros(want, g, bits), q.AdamWTensors.zeros(p, g, bits)
    for plan in (plain, dropped):
        q.adamw_step_many(plan, lr=1e-2, step=1, seed=3)
    q.adamw_step_many(plain, lr=1e-2, step=2, seed=4)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(2000000)
        q.adamw_step_many(dropped, lr=1e-2, step=2, seed=4)
        del dropped, plan
    scribble = [torch.full((n * (4 if bits == 32 else 1),), 0x77, dtype=torch.uint8, device=DEV) for n in sizes * 2]
    scribble += [torch.full((-(-n // 256),), 1e9, device=DEV) for n in sizes * 2]
    stream.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(p, want):
        assert torch.equal(x, y)
    assert all(bool((x == (0x77 if x.dtype == torch.uint8 else 1e9)).all()) for x in scribble)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_launches_captured(bits):
    """A captured step of more tensors than a launch takes, replayed with eager steps of another object between the
    replays, gives what they give; only the gradients and their factor are read anew."""
    print(f"adamw launches captured {bits}", flush=True)
    sizes = [(53 * i) % 700 for i in range(1100)]
    a, b = Many(sizes, "bf16", "bf16", bits, 71), Many(sizes, "bf16", "bf16", bits, 71)
    scale = torch.full((1,), 0.5, device=DEV)
    step = lambda t: q.adamw_step_many(t.plan, lr=1e-3, step=7, grad_scale=scale, seed=8)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(a)
    for rep in range(3):
        step(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("dp", "dm", "dv", "copy") + (("dms", "dvs") if bits == 8 else ()):
            for x, y in zip(getattr(a, name), getattr(b, name)):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (rep, name)
        scale.fill_(0.25)
        for x, y in zip(a.dg, b.dg):
            x.neg_()
            y.neg_()
