"""AdamW over parameters that have taken different numbers of steps: each is stepped as it
would be alone. And which tensors of an optimizer may be replaced."""
import numpy as np
import pytest
import torch

gpu = pytest.mark.gpu
HY = dict(lr=3e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.1)


def _run(opt_of, sizes, dtype, steps, skip, seed=0):
    """One optimizer over all, and one of each parameter alone, the same gradients."""
    g = torch.Generator().manual_seed(seed)
    ps = [(torch.randn(n, generator=g) * 0.02).to(dtype).cuda() for n in sizes]
    joint, alone = opt_of([p.clone() for p in ps]), [opt_of([p.clone()]) for p in ps]
    for t in range(steps):
        grads = [None if skip(t, i) else (torch.randn(n, generator=g) * 1e-2).to(dtype).cuda()
                 for i, n in enumerate(sizes)]
        joint.step(grads)
        for one, gr in zip(alone, grads):
            if gr is not None:
                one.step([gr])
    return joint, alone


@gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,master", [(torch.float32, None), (torch.bfloat16, None), (torch.bfloat16, True)])
@pytest.mark.parametrize("sizes", [[5, 300, 2049], [(i * 37) % 300 + 1 for i in range(450)]],
                         ids=["three", "many"])
def test_each_as_it_would_be_alone(bits, dtype, master, sizes):
    from lm_head_jsd_gb300 import AdamW

    def skip(t, i):  # 0: never, 1: from the third step on, 2: every other step
        return i % 3 == 1 and t < 3 or i % 3 == 2 and t % 2 == 1

    joint, alone = _run(lambda ps: AdamW(ps, state_bits=bits, master=master, **HY), sizes, dtype, 5, skip)
    for name in ("params", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        if getattr(joint, name) is not None:
            for a, one in zip(getattr(joint, name), alone):
                assert torch.equal(a.float(), getattr(one, name)[0].float()), name
    assert joint.steps == 5 and joint.param_steps == [one.steps for one in alone]


@gpu
def test_late_parameter_against_torch():
    from lm_head_jsd_gb300 import AdamW

    g = torch.Generator().manual_seed(1)
    start = [torch.randn(40, generator=g) for _ in range(2)]
    ours = AdamW([p.cuda() for p in start], **HY)
    ref = [torch.nn.Parameter(p.double()) for p in start]
    theirs = torch.optim.AdamW(ref, **HY)
    for t in range(60):
        grads = [torch.randn(40, generator=g), torch.randn(40, generator=g) if t >= 50 else None]
        ours.step([None if x is None else x.cuda() for x in grads])
        for p, x in zip(ref, grads):
            p.grad = None if x is None else x.double()
        theirs.step()
    # each step: two roundings of p and six of an update of at most lr (1 + a few)
    lim = 60 * (2 ** -23 * 5 + 2 ** -21 * 4 * HY["lr"])
    for a, b in zip(ours.params, ref):
        assert (a.cpu().double() - b.detach()).abs().max().item() <= lim
    assert ours.steps == 60 and ours.param_steps == [60, 10]


@gpu
def test_counts_go_on_from_a_checkpoint():
    from lm_head_jsd_gb300 import AdamW

    sizes = [129, 300, 7]
    opt = lambda ps, **kw: AdamW(ps, state_bits=8, **HY, **kw)  # noqa: E731
    joint, _ = _run(opt, sizes, torch.float32, 4, lambda t, i: i == 1 and t != 2)
    again = opt([p.clone() for p in joint.params], exp_avg=[t.clone() for t in joint.exp_avg],
                exp_avg_sq=[t.clone() for t in joint.exp_avg_sq],
                exp_avg_scale=[t.clone() for t in joint.exp_avg_scale],
                exp_avg_sq_scale=[t.clone() for t in joint.exp_avg_sq_scale], step=joint.param_steps)
    assert again.param_steps == [4, 1, 4] and again.steps == 4
    grads = [torch.ones(n, device="cuda") for n in sizes]
    joint.step(grads)
    again.step(grads)
    assert all(torch.equal(a, b) for a, b in zip(joint.params, again.params))
    assert joint.param_steps == again.param_steps == [5, 2, 5]


def test_counts_without_a_gpu():
    from lm_head_jsd_gb300 import AdamW

    p = [torch.zeros(4), torch.zeros(3)]
    assert AdamW(p).param_steps == [0, 0]
    assert AdamW(p, step=7).param_steps == [7, 7]
    assert AdamW(p, step=[7, 2]).param_steps == [7, 2] and AdamW(p, step=(7, 2)).steps == 7
    assert AdamW(p, step=np.array([3, 3])).param_steps == [3, 3]
    for bad in ([1], [1, 2, 3], [[1, 2]]):
        with pytest.raises(ValueError):
            AdamW(p, step=bad)


def test_states_are_not_replaced():
    """The kernel's table holds the addresses of the tensors of the construction: another
    tensor in their place would be left as it is, and the old one's memory written when it
    may be another's."""
    from lm_head_jsd_gb300 import AdamW

    p = [torch.zeros(4).bfloat16(), torch.zeros(300).bfloat16()]
    opt = AdamW(p, state_bits=8, master=True)
    for name in ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        ts = getattr(opt, name)
        with pytest.raises(TypeError):
            ts[0] = ts[0].clone()
        with pytest.raises(AttributeError):
            setattr(opt, name, [t.clone() for t in ts])
        ts[0].view(torch.uint8).zero_()  # (contents may be written)


@gpu
def test_replaced_parameters_and_storages():
    from lm_head_jsd_gb300 import AdamW

    g = torch.ones(300, device="cuda")
    opt = AdamW([torch.ones(300, device="cuda") for _ in range(2)], **HY)
    ref = AdamW([torch.ones(300, device="cuda") for _ in range(2)], **HY)
    opt.step([g, g])
    ref.step([g, g])
    old = opt.params[0]
    opt.params[0] = old.clone()  # another tensor in a parameter's place is stepped
    kept, version = old.clone(), opt.params[0]._version
    opt.step([g, g])
    ref.step([g, g])
    assert torch.equal(opt.params[0], ref.params[0]) and torch.equal(old, kept)
    assert opt.params[0]._version > version
    # a state whose storage is replaced: the old memory is still the optimizer's own
    at = opt.exp_avg[0].data_ptr()
    opt.exp_avg[0].data = opt.exp_avg[0].clone()
    later = [torch.full((300,), 5.0, device="cuda") for _ in range(20)]
    assert at not in [t.data_ptr() for t in later]
    opt.step([g, g])
    torch.cuda.synchronize()
    assert all((t == 5).all() for t in later)


@gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_every_count_another(bits):
    """Parameters of as many counts as there are: each as alone, in two launches for 450."""
    from lm_head_jsd_gb300 import AdamW, fljsd_launch_count

    sizes = [(i * 53) % 400 + 1 for i in range(450)]
    g = torch.Generator().manual_seed(3)
    ps = [torch.randn(n, generator=g).cuda() for n in sizes]
    gs = [torch.randn(n, generator=g).cuda() for n in sizes]
    joint = AdamW([p.clone() for p in ps], state_bits=bits, step=list(range(450)), **HY)
    before = fljsd_launch_count()
    joint.step(gs)
    assert fljsd_launch_count() - before == 2
    for i, (p, q) in enumerate(zip(ps, joint.params)):
        one = AdamW([p.clone()], state_bits=bits, step=i, **HY)
        one.step([gs[i]])
        assert torch.equal(one.params[0], q), i


def test_counts_that_are_refused():
    import ctypes

    from conftest import build_library

    build_library()
    from lm_head_jsd_gb300 import _lib as L

    o = L.make_adamw_options(1e-3, 0.9, 0.99, 1e-8, 0.0, 0)  # (its own step is not used)
    t = (L.fljsd_adamw_tensor * 2)()
    call = lambda *steps: L.fljsd_adamw_step_each(  # noqa: E731
        o, ctypes.addressof(t), ctypes.addressof((ctypes.c_int64 * 2)(*steps)), 2, None, stream=0, check=False)
    assert call(1, 1) == 0  # two tensors without elements: nothing to do
    assert call(1, 0) == 1 and call(-3, 1) == 1
    assert L.fljsd_adamw_step_each(o, ctypes.addressof(t), None, 2, None, stream=0, check=False) == 1
