"""The training operators on streams other than their tensors' own."""
import pytest
import torch

import train_ref as R
from sparse_moe_ffn_gemv_b200 import train
from test_train_ops import gen, ok, planes, rand, spec_of

pytestmark = pytest.mark.gpu


def calls():
    """(operator, name, tensors, call of copies of the tensors on a stream)"""
    g = gen(71)
    T, H, N = 517, 1032, 776
    x, w, b = rand(g, (T, H), "bf16"), rand(g, (N, H), "bf16", H ** -0.5), rand(g, (N,), "bf16")
    r, pre = rand(g, (T, N), "bf16"), rand(g, (T, N), "bf16")
    lin, norm = train.Linear(H, N, activation="silu"), train.Norm(H, kind="layer")
    gamma = rand(g, (H,), "bf16", 0.3, 1.0)
    stats = norm.forward(x, gamma)[1]
    dy = rand(g, (T, H), "bf16")
    spec = spec_of(num_experts=3, top_k=2, hidden=H, intermediate=264, has_expert_bias=True)
    p = planes(spec, g)
    names, values = list(p), list(p.values())
    off, slots, wts = R.make_routing(T, spec, g, "cuda")
    fpre = rand(g, (2 * T, 528), "bf16")
    ffn = train.GatedFfn(spec)
    plane = lambda v: dict(zip(names, v))  # noqa: E731
    return [
        (lin, "linear", [x, w, b, r], lambda t, s: lin.forward(t[0], t[1], bias=t[2], residual=t[3], stream=s)),
        (lin, "linear backward", [r, x, w, pre], lambda t, s: lin.backward(*t[:3], pre=t[3], stream=s)),
        (norm, "norm", [x, gamma, gamma], lambda t, s: norm.forward(t[0], t[1], bias=t[2], stream=s)),
        (norm, "norm backward", [dy, x, gamma, stats], lambda t, s: norm.backward(*t, stream=s)),
        (ffn, "ffn", [x, off, slots, wts] + values,
         lambda t, s: ffn.forward(t[0], plane(t[4:]), routing=tuple(t[1:4]), residual=t[0], stream=s)),
        (ffn, "ffn backward", [dy, x, fpre, off, slots, wts] + values,
         lambda t, s: list(ffn.backward(*t[:2], plane(t[6:]), t[2], routing=tuple(t[3:6]), stream=s).values())),
    ]


def test_tensors_may_be_dropped_behind_a_call_on_a_stream():
    """Inputs that go out of scope while the stream of the call is still busy with something else are
    not handed out again to the caller's stream."""
    s = torch.cuda.Stream()
    for op, name, tensors, call in calls():
        flat = lambda o: [o] if torch.is_tensor(o) else list(o)  # noqa: E731
        want = flat(call(tensors, torch.cuda.current_stream()))
        copies = [t.clone() for t in tensors]
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)  # about 50 ms
        got = flat(call(copies, s))
        del copies
        # what the caller's stream allocates next, and fills
        again = [torch.zeros_like(t) for t in tensors for _ in range(3)]
        ok(op)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name
        del again


def test_a_stream_of_another_operators_results():
    """A chain over two named streams with waits between them."""
    g = gen(72)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    x, w = rand(g, (300, 264), "bf16"), rand(g, (264, 264), "bf16", 0.06)
    op = train.Linear(264, 264, activation="gelu")
    want = op.forward(op.forward(op.forward(x, w), w), w)
    a.wait_stream(torch.cuda.current_stream())
    y = op.forward(x, w, stream=a)
    b.wait_stream(a)
    z = op.forward(y, w, stream=b)
    a.wait_stream(b)
    del y
    z = op.forward(z, w, stream=a)
    torch.cuda.current_stream().wait_stream(a)
    ok(op)
    assert torch.equal(z, want)


def test_captured_on_a_named_stream():
    """Calls that name the stream which a graph is captured on, with tensors of another stream."""
    s = torch.cuda.Stream()
    for op, name, tensors, call in calls():
        flat = lambda o: [o] if torch.is_tensor(o) else list(o)  # noqa: E731
        want = flat(call(tensors, torch.cuda.current_stream()))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = flat(call(tensors, s))
        for _ in range(2):
            for t in got:
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            ok(op)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name


def test_external_stream():
    """A stream that PyTorch did not make runs the calls, and no tensor is recorded on it: it may be
    gone when the tensor is freed."""
    inner = torch.cuda.Stream()
    s = torch.cuda.ExternalStream(inner.cuda_stream)
    recorded = []

    class Marked(torch.Tensor):
        def record_stream(self, stream):
            recorded.append(stream)
            super().record_stream(stream)

    for op, name, tensors, call in calls():
        flat = lambda o: [o] if torch.is_tensor(o) else list(o)  # noqa: E731
        want = flat(call(tensors, torch.cuda.current_stream()))
        torch.cuda.synchronize()
        got = flat(call([t.as_subclass(Marked) for t in tensors], s))
        ok(op)
        assert all(torch.equal(a.as_subclass(torch.Tensor), b) for a, b in zip(got, want)), name
        assert not recorded
    lin, _, tensors, call = calls()[0]
    call([t.as_subclass(Marked) for t in tensors], inner)
    ok(lin)
    assert len(recorded) == len(tensors)
