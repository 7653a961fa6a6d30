"""The binding's own checks of the microscaled operators and the optimiser, on
stand-ins: CPU tensors that call themselves GPU tensors, with the library's entry
points replaced (CPU only: no kernel is ever launched here)."""

import pytest

tw = pytest.importorskip("activation_sparse_transformer_bf16_amd")
torch = pytest.importorskip("torch")

DEVICE = torch.device("cuda:0")


class OnGpu(torch.Tensor):
    is_cuda = property(lambda self: True)
    device = property(lambda self: DEVICE)


def gpu(t):
    return t.as_subclass(OnGpu)


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The entry points called, in place of the calls."""
    seen = []
    monkeypatch.setattr(tw, "_launch", lambda device, fn, *args: seen.append(args))
    return seen


def rows(q, scale, cols, factor=None):
    return tw.Mx4Rows(gpu(q), gpu(scale), cols, factor)


def _one_row_views():
    """(q, scale, columns) of one row whose elements do not lie next to one another."""
    q, scale = torch.zeros(1, 32, dtype=torch.uint8), torch.zeros(1, 16, dtype=torch.uint8)
    yield torch.zeros(1, 64, dtype=torch.uint8)[:, ::2], scale, 64
    yield q, torch.zeros(1, 32, dtype=torch.uint8)[:, ::2], 64
    yield torch.zeros(1, 1, dtype=torch.uint8).expand(1, 4096), torch.zeros(1, 256, dtype=torch.uint8), 8192
    yield q, torch.zeros(1, 1, dtype=torch.uint8).expand(1, 16), 64


@pytest.mark.parametrize("view", range(4))
def test_a_single_row_has_unit_stride(view, calls):
    q, scale, cols = list(_one_row_views())[view]
    bad = rows(q, scale, cols)
    x = gpu(torch.zeros(1, cols))
    factor = gpu(torch.zeros(1))
    good = rows(torch.zeros(1, cols // 2, dtype=torch.uint8), torch.zeros(1, -(-cols // 512) * 16, dtype=torch.uint8), cols)
    for call in (lambda: tw.twell_quantize_mx4(x, out=bad), lambda: tw.twell_dequantize_mx4(bad, y=x),
                 lambda: tw.twell_rmsnorm_mx4(x, x[0], h=x, y=x, q=tw.Mx4Rows(bad.q, bad.scale, cols, factor)),
                 lambda: tw.twell_mx4_matmul(bad, good, y=gpu(torch.zeros(1, 1))),
                 lambda: tw.twell_mx4_matmul(good, bad, y=gpu(torch.zeros(1, 1)))):
        with pytest.raises(ValueError, match="unit stride"):
            call()
    assert not calls


def test_a_single_row_of_any_row_stride(calls):
    # a row's own stride to the next one says nothing where there is none; a single byte has no stride along
    wide = torch.zeros(3, 40, dtype=torch.uint8)
    one = rows(wide[1:2, :32], torch.zeros(1, 16, dtype=torch.uint8).as_strided((1, 16), (7, 1)), 64)
    tw.twell_quantize_mx4(gpu(torch.zeros(1, 64)), out=one)
    byte = rows(torch.zeros(1, 16, dtype=torch.uint8).as_strided((1, 1), (16, 5)), torch.zeros(1, 16, dtype=torch.uint8), 2)
    tw.twell_quantize_mx4(gpu(torch.zeros(1, 2)), out=byte)
    assert len(calls) == 2


def test_the_sizes_of_rows_are_fixed(calls):
    # the library's rows lie in one buffer of exactly that many
    made = tw.Mx4Rows.empty(3, 64, "cpu")
    given = rows(torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(3, 16, dtype=torch.uint8), 64)
    for r in (made, given):
        for name in ("rows", "cols", "q", "scale", "factor"):
            with pytest.raises(AttributeError):
                setattr(r, name, 1000)
        assert (r.rows, r.cols) == (3, 64) and r.q.shape == (3, 32) and r.scale.shape == (3, 16)


def optimizer(bits=8, sizes=(40, 50)):
    """(optimiser, gradients) of float32 weights."""
    zeros = [gpu(torch.zeros(n)) for n in sizes]
    blocks = [-(-n // 32) for n in sizes]
    states = [[gpu(torch.zeros(n, dtype=torch.uint8 if bits == 8 else torch.float32)) for n in sizes] for _ in range(2)]
    scales = [[gpu(torch.zeros(n, dtype=torch.uint8)) for n in blocks] if bits == 8 else None for _ in range(2)]
    return tw.TwellAdamW(zeros, *states, *scales), [gpu(torch.ones(n)) for n in sizes]


def step(opt, grads):
    tw.twell_adamw_step(opt, grads, lr=1e-3, step=1)


def _listed(call, opt, field):
    """A field of twell_adamw_tensor in the list that a call passed."""
    table = (tw.TwellAdamWTensorC * len(opt.weights)).from_buffer_copy(call[0])
    return [getattr(t, field) for t in table]


# what a resumed run may put in the place of the states: on the host, too short, of another type, too few, none
BAD_STATES = [lambda a: [t.as_subclass(torch.Tensor) for t in a], lambda a: [a[0], a[1][:49]], lambda a: [t.short() for t in a],
              lambda a: a[:1], lambda a: None, lambda a: [a[0], None], lambda a: [a[0], a[0]]]


@pytest.mark.parametrize("name", ["m", "v", "m_scale", "v_scale"])
@pytest.mark.parametrize("bad", range(len(BAD_STATES)))
def test_states_put_in_place_are_checked(name, bad, calls):
    opt, grads = optimizer()
    step(opt, grads)
    good = getattr(opt, name)
    setattr(opt, name, [good[0], good[1][:1]] if name.endswith("scale") and bad == 1 else BAD_STATES[bad](list(good)))
    for call in (lambda: step(opt, grads), lambda: tw.twell_adamw_states(opt)) * 2:  # refused again, not once
        with pytest.raises((ValueError, TypeError)):
            call()
    assert len(calls) == 1
    setattr(opt, name, [t.clone() for t in good])
    step(opt, grads)
    assert _listed(calls[-1], opt, name) == [t.data_ptr() for t in getattr(opt, name)]
    assert getattr(opt, name)[0].data_ptr() != good[0].data_ptr()


@pytest.mark.parametrize("bits", [32, 8])
def test_states_given_other_storage_are_checked(bits, calls):
    for name in ("m", "v"):
        opt, grads = optimizer(bits)
        t = getattr(opt, name)[1]
        t.data = torch.zeros(50, dtype=t.dtype)
        step(opt, grads)
        assert _listed(calls[-1], opt, name)[1] == t.data_ptr()
        t.data = torch.zeros(49, dtype=t.dtype)
        with pytest.raises(ValueError):
            step(opt, grads)
        # fewer elements of the same memory; memory that was given back
        opt, grads = optimizer(bits)
        t = getattr(opt, name)[1]
        t.data = t.data[:49]
        with pytest.raises(ValueError):
            step(opt, grads)
        opt, grads = optimizer(bits)
        getattr(opt, name)[1].untyped_storage().resize_(0)
        with pytest.raises(ValueError, match="storage"):
            step(opt, grads)


def test_decay_put_in_place(calls):
    opt, grads = optimizer()
    opt.weight_decay = 0.5
    step(opt, grads)
    assert _listed(calls[-1], opt, "weight_decay") == [0.5, 0.5]
    opt.weight_decay = [0.25]
    with pytest.raises(ValueError):
        step(opt, grads)


def test_weights_given_other_storage_are_checked(calls):
    opt, grads = optimizer()
    a, b = opt.weights
    b.data = torch.zeros(50)  # as a module's own conversions do
    step(opt, grads)
    assert _listed(calls[-1], opt, "weight") == [a.data_ptr(), b.data_ptr()]
    # side by side in one buffer; then one over the other
    whole = torch.zeros(90)
    a.data, b.data = whole[:40], whole[40:]
    step(opt, grads)
    b.data = whole[39:89]
    for _ in range(2):
        with pytest.raises(ValueError, match="share memory"):
            step(opt, grads)
    for bad, error in ((torch.zeros(50).bfloat16(), TypeError), (torch.zeros(51), ValueError), (torch.zeros(100)[::2], ValueError)):
        opt, grads = optimizer()
        opt.weights[1].data = bad
        for _ in range(2):
            with pytest.raises(error):
                step(opt, grads)
    opt, grads = optimizer()
    opt.weights = [gpu(torch.zeros(40)), gpu(torch.zeros(51))]
    with pytest.raises(ValueError):
        step(opt, grads)


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_in_written_memory_are_refused(bits, calls):
    # a step reads them while it writes the others
    whole = torch.zeros(1000)
    w = [gpu(whole[100:140]), gpu(whole[140:190])]  # side by side
    opt, _ = optimizer(bits)
    opt.weights = w
    fine = [gpu(whole[60:100]), gpu(whole[190:240])]  # up to their first byte and from their last on
    step(opt, fine)
    step(opt, [gpu(whole[300:340]), gpu(whole[290:340])])  # each other's memory, which is only read
    assert _listed(calls[-1], opt, "grad") == [whole[300:].data_ptr(), whole[290:].data_ptr()]
    half = whole.view(torch.bfloat16)
    step(opt, [gpu(half[160:200]), gpu(half[380:430])])
    states = [t for name in ("m", "v", "m_scale", "v_scale") for t in getattr(opt, name) if t is not None]
    inside = [whole[61:101], whole[100:140], whole[101:141], whole[139:179], whole[150:190], whole[189:229],
              half[161:201], half[379:419]]
    for one in inside:
        with pytest.raises(ValueError, match="share memory"):
            step(opt, [gpu(one), fine[1]])
    for t in states:
        if t.dtype == torch.float32 and t.numel() == 40:
            with pytest.raises(ValueError, match="share memory"):
                step(opt, [t, fine[1]])
    if bits == 8:  # bytes of codes, as an element of a gradient
        one, grads = optimizer(8, (4, 1))
        with pytest.raises(ValueError, match="share memory"):
            step(one, [grads[0], gpu(one.m[0].as_subclass(torch.Tensor).view(torch.float32))])
    n = len(calls)
    # a tensor without elements lies nowhere
    opt, grads = optimizer(bits, (0, 40, 0))
    opt.weights = [opt.weights[0], opt.weights[1], gpu(opt.weights[1].as_subclass(torch.Tensor)[:0])]
    grads[2] = gpu(opt.weights[1].as_subclass(torch.Tensor)[20:20])
    step(opt, grads)
    assert len(calls) == n + 1


def test_gradients_in_the_copies_are_refused(calls):
    w = gpu(torch.zeros(64, dtype=torch.bfloat16))
    opt = tw.TwellAdamW([w], [gpu(torch.zeros(64))], [gpu(torch.zeros(64))], master=[gpu(torch.zeros(64))])
    step(opt, [gpu(torch.zeros(64))])
    for grad in (opt.master[0], opt.m[0], opt.v[0], w):
        with pytest.raises(ValueError, match="share memory"):
            step(opt, [grad])
    assert len(calls) == 1


def test_autograd_sees_the_step(calls):
    # a backward through a graph of the weights before the step would use those after it
    w = gpu(torch.full((40,), 2.0)).requires_grad_()
    b = gpu(torch.zeros(40, dtype=torch.bfloat16))
    with torch.inference_mode():
        i = gpu(torch.zeros(40))  # has no version
    copy = gpu(torch.zeros(40))
    zeros = lambda: [gpu(torch.zeros(40)) for _ in range(3)]  # noqa: E731
    opt = tw.TwellAdamW([w, b, i], zeros(), zeros(), master=[None, copy, None])
    loss, later = (w * w).sum(), (w * 3).sum()
    before = w._version, b._version, copy._version
    step(opt, zeros())
    assert all(t._version > v for t, v in zip((w, b, copy), before)) and len(calls) == 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    later.backward()  # needs no weight
    assert torch.equal(w.grad.as_subclass(torch.Tensor), torch.full((40,), 3.0))
    # a refused step has written nothing
    before = w._version
    with pytest.raises(ValueError):
        tw.twell_adamw_step(opt, zeros(), lr=1e-3, step=0)
    assert w._version == before


def test_the_quantiser_refuses_rows_beyond_32_bits(calls):
    # (ctypes would pass their low 32 bits); without memory, but on the GPU as far as the checks can tell
    for shape in (((1 << 31) + 3, 32), (3, 1 << 31)):
        x = gpu(torch.empty(shape, dtype=torch.bfloat16, device="meta"))
        for call in (lambda: tw.twell_quantize_mx4(x), lambda: tw.twell_rmsnorm_mx4(x, gpu(torch.empty(shape[1], device="meta")))):
            with pytest.raises(ValueError, match=f"sizes of .*{max(shape)}.* exceed"):
                call()
    small = gpu(torch.zeros(3, 32))
    tw.twell_quantize_mx4(small, out=rows(torch.zeros(3, 16, dtype=torch.uint8), torch.zeros(3, 16, dtype=torch.uint8), 32))
    assert len(calls) == 1


def test_storage_given_back_is_refused(calls):
    # as a sharded module gives back its flat buffer between steps; a view's address is then small and not 0
    flat = torch.zeros(200)
    opt, grads = optimizer(8, (40, 50))
    opt.weights = [gpu(flat[100:140]), gpu(flat[140:190])]
    step(opt, grads)
    flat.untyped_storage().resize_(0)
    for _ in range(2):
        with pytest.raises(ValueError, match="given back"):
            step(opt, grads)
    assert len(calls) == 1
    flat.untyped_storage().resize_(800)
    step(opt, grads)
    assert _listed(calls[-1], opt, "weight") == [flat[100:].data_ptr(), flat[140:].data_ptr()]


class Elsewhere(OnGpu):
    device = property(lambda self: torch.device("cuda:1"))


def test_an_optimiser_moved_to_another_device(monkeypatch):
    seen = []
    monkeypatch.setattr(tw, "_launch", lambda device, fn, *args: seen.append(device))
    opt, grads = optimizer(32)
    step(opt, grads)
    for name in ("weights", "m", "v"):
        setattr(opt, name, (t.as_subclass(Elsewhere) for t in getattr(opt, name)))  # (any iterable)
    lr = torch.zeros(1).as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        step(opt, grads)
    there = [g.as_subclass(Elsewhere) for g in grads]
    with pytest.raises(ValueError):
        tw.twell_adamw_step(opt, there, lr=gpu(torch.zeros(1)), step=1)
    tw.twell_adamw_step(opt, there, lr=lr, step=1)
    assert seen == [torch.device("cuda:0"), torch.device("cuda:1")]
