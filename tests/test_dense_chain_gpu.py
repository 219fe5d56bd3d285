"""The dense calls together, as a decoder layer makes them: in the example stack with 8-bit
projections and rotary positions (every call against fp64 on the inputs that it got), captured
into graphs, and on other streams."""
import numpy as np
import pytest
import torch

import dense_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda
from test_hybrid_example_gpu import _example

pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def _value(codes, scales, rows):
    return ref.value(codes.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), rows)


def test_every_call_of_the_8_bit_stack(monkeypatch):
    ex = _example()
    calls = []
    for name in ("kda_add_rmsnorm_fp8", "kda_fp8_quant", "kda_fp8_matmul", "kda_rotary"):
        def record(*args, _f=getattr(kda, name), _name=name, **kw):
            before = [a.clone() if isinstance(a, torch.Tensor) else a for a in args]
            out = _f(*args, **kw)
            calls.append((_name, before, tuple(o.clone() if o is not None else None for o in (out if isinstance(out, tuple) else (out,)))))
            return out
        monkeypatch.setattr(kda, name, record)
    model = ex.HybridDecoder(3, 160, page_size=16, fp8=True, rotary_base=10000.0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    calls.clear()   # the weights' quantisation has its own tests
    positions = [0, 0, 0]
    for take in ([70, 0, 33], [2, 40, 1], [1, 1, 1], [1, 1, 1]):
        y = model.step(torch.randn(sum(take), 512, device="cuda", generator=gen).bfloat16(), take)
        assert torch.isfinite(y.float()).all() and y.shape == (sum(take), 512)
        want = np.concatenate([np.arange(p, p + t) for p, t in zip(positions, take)])
        turned = [c for c in calls if c[0] == "kda_rotary"]
        assert len(turned) == 1 and np.array_equal(turned[0][1][2].cpu().numpy(), want)   # the page map's positions
        positions = [p + t for p, t in zip(positions, take)]
        assert [c[0] for c in calls].count("kda_fp8_matmul") == 8 and [c[0] for c in calls].count("kda_add_rmsnorm_fp8") == 4
        for name, args, out in calls:
            if name == "kda_add_rmsnorm_fp8":
                s, y64 = ref.norm(f64(args[0]), f64(args[1]) if len(args) > 1 else None, None, np.float64(np.float32(1e-6)))
                near = 1 + 32 * 2.0 ** -24   # as for the norm alone
                b = out[1].cpu().numpy()
                assert ((b >= ref.scale_bytes(y64 / near, 1)) & (b <= ref.scale_bytes(y64 * near, 1))).all()
                unit = np.ldexp(1.0, ref.per_element(b, 1, *y64.shape) - 127)
                step = np.ldexp(1.0, np.maximum(np.frexp(np.abs(y64) * near / unit)[1] - 1, -6) - 3) * unit
                assert (np.abs(_value(out[0], out[1], 1) - y64) <= 0.5 * step + 32 * 2.0 ** -24 * np.abs(y64)).all()
                if len(args) > 1:
                    assert torch.equal(out[2], (args[0].float() + args[1].float()).bfloat16())
            elif name == "kda_fp8_quant":
                c, b = ref.stored(f64(args[0]), 1)
                assert np.array_equal(out[0].view(torch.uint8).cpu().numpy(), c) and np.array_equal(out[1].cpu().numpy(), b)
            elif name == "kda_fp8_matmul":
                a, w = _value(args[0], args[1], 1), _value(args[2], args[3], 128)
                want, size = a @ w.T, np.abs(a) @ np.abs(w).T
                tol = (a.shape[1] / 32 + 8) * 2.0 ** -22 * size + 2.0 ** -8 * np.abs(want)
                assert (np.abs(f64(out[0]) - want) <= tol).all()
            else:
                pos, freqs = args[2].cpu().numpy(), args[3].cpu().numpy()
                for x, o in zip(args[:2], out):
                    want = ref.rotate(f64(x), pos, freqs, 1.0, False, False)
                    size = 2 * np.abs(f64(x)).max(-1, keepdims=True)
                    assert (np.abs(f64(o) - want) <= 2.0 ** -20 * size + 2.0 ** -8 * np.abs(want)).all()
        calls.clear()
    assert kda.kda_device_error() == (0, 0)


def test_example_runs_in_8_bits(capsys):
    x = _example().main(4, 100, 3, 1)
    assert torch.isfinite(x.float()).all()
    assert "pages in use" in capsys.readouterr().out


class Layer:
    """The dense half of an attention layer on inputs that stay where they are."""

    def __init__(self, T, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x, self.res = (torch.randn(T, 512, device="cuda", generator=g).bfloat16() for _ in range(2))
        self.w = kda.kda_fp8_quant(torch.randn(8 * 128, 512, device="cuda", generator=g), 128)
        self.pos = torch.randint(0, 1000, (T,), device="cuda", generator=g).to(torch.int32)
        self.freqs, _ = kda.kda_rotary_freqs(128)

    def __call__(self, **kw):
        codes, scales, h = kda.kda_add_rmsnorm_fp8(self.x, self.res, **kw)
        p = kda.kda_fp8_matmul(codes, scales, *self.w, **kw)
        q, k = p[:, :768].unflatten(1, (6, 128)), p[:, 768:].unflatten(1, (2, 128))
        kda.kda_rotary(q, k, self.pos, self.freqs, q_out=q, k_out=k, **kw)
        return h, p, kda.kda_fp8_values(*kda.kda_fp8_quant(p, **kw), **kw)


@pytest.mark.parametrize("T", [1, 77, 700])
def test_captured_into_graphs(T):
    """Two graphs of the same calls, replayed in turn with new inputs, give what the calls give."""
    layers = [Layer(T, 1), Layer(T, 2)]
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for layer in layers:
            layer()
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = layer()
            graphs.append((g, out))
    for i in range(3):
        for layer, (g, out) in zip(layers, graphs):
            layer.x.copy_(torch.randn_like(layer.x))
            layer.pos.add_(17)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, layer()):
                assert torch.equal(a, b)
    assert kda.kda_device_error() == (0, 0)


def test_on_another_stream():
    """A stream given by object or handle: the work, and the memory of the results, belong to it."""
    layer = Layer(300, 3)
    want = layer()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = layer(stream=stream)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_calls_in_flight_at_once():
    """The same calls on four streams at once, without scratch memory to share."""
    layers = [Layer(t, 10 + t) for t in (1, 64, 300, 1500)]
    want = [layer() for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    got = []
    for _ in range(5):
        got.append([])
        for layer, s in zip(layers, streams):
            with torch.cuda.stream(s):
                got[-1].append(layer())
    torch.cuda.synchronize()
    for round_ in got:
        for outs, ws in zip(round_, want):
            for a, b in zip(outs, ws):
                assert torch.equal(a, b)


def test_one_behind_another():
    """300 dependent steps without a wait between them (a residual stream updated in place, an input that each step's
    product writes) give the bits that they give with the GPU waited for after every call."""
    def run(wait):
        g = torch.Generator(device="cuda").manual_seed(5)
        res = torch.randn(200, 512, device="cuda", generator=g).bfloat16()
        w = kda.kda_fp8_quant(torch.randn(512, 512, device="cuda", generator=g) * 0.05, 128)
        x, pos = torch.zeros_like(res), torch.arange(200, device="cuda", dtype=torch.int32)
        freqs, _ = kda.kda_rotary_freqs(64)
        for i in range(300):
            codes, scales, _ = kda.kda_add_rmsnorm_fp8(x, res, residual_out=res)
            wait()
            kda.kda_fp8_matmul(codes, scales, *w, out=x)
            wait()
            heads = x.view(200, 8, 64)
            kda.kda_rotary(heads, None, pos, freqs, q_out=heads)
            wait()
            if i % 7 == 0:
                x.copy_(kda.kda_fp8_values(*kda.kda_fp8_quant(x, 128), 128))
                wait()
        return res, x

    for a, b in zip(run(lambda: None), run(torch.cuda.synchronize)):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)
