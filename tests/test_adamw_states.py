"""What AdamW does when its states are replaced, as a loaded checkpoint's are:
the next step works on the new ones, or refuses.  Without a GPU the call's
list is read instead of run."""
import pytest
import torch

import sparse_mixture_experts_50_amd as moe
import sparse_mixture_experts_50_amd.optim as optim_module

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture
def calls(monkeypatch):
    """One entry for each launched step: the list's addresses, by name."""
    seen = []

    def run(name, device, h, n, tensors):
        seen.append([{f: getattr(t, f) for f, _ in t._fields_}
                     for t in tensors])

    monkeypatch.setattr(optim_module, "_run", run)
    return seen


def optimizer(bits):
    opt = moe.AdamW([torch.zeros(40), torch.zeros(3, 5, dtype=BF)], lr=1.0,
                    state_bits=bits, master=True)
    return opt, [torch.zeros(40), torch.zeros(3, 5)]


def lists(opt):
    names = ["m", "v", "master"]
    return names + (["m_scale", "v_scale"] if opt.state_bits == 8 else [])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_replaced_state_is_the_next_steps(bits, calls):
    opt, grads = optimizer(bits)
    opt.step(grads)
    for name in lists(opt):
        # an entry, its memory, the whole list
        own = getattr(opt, name)
        own[1] = own[1].clone()
        opt.step(grads)
        assert calls[-1][1][name] == own[1].data_ptr(), name
        own[1].data = own[1].clone()
        opt.step(grads)
        assert calls[-1][1][name] == own[1].data_ptr(), name
        setattr(opt, name, [None if t is None else t.clone() for t in own])
        opt.step(grads)
        for i, t in enumerate(getattr(opt, name)):
            assert calls[-1][i][name] == (None if t is None
                                          else t.data_ptr()), name
    assert opt.steps == 1 + 3 * len(lists(opt)) == len(calls)


@pytest.mark.parametrize("bits", [32, 8])
def test_what_cannot_be_a_state_is_refused(bits, calls):
    opt, grads = optimizer(bits)
    for name in lists(opt):
        own = getattr(opt, name)
        good, dtype = own[1], own[1].dtype
        other = BF if dtype == F32 else F32
        rows = torch.zeros(good.numel() * 2, dtype=torch.uint8)
        for bad in (None, good.clone().view(-1)[:-1].clone(),
                    torch.zeros(good.shape, dtype=other),
                    torch.zeros(good.shape, dtype=dtype, device="meta"),
                    torch.empty((*good.shape, 2), dtype=dtype)[..., 0]
                    if good.numel() > 1 else rows, 0.5):
            own[1] = bad
            with pytest.raises((ValueError, AttributeError)):
                opt.step(grads)
            own[1] = good
        own.append(good)
        with pytest.raises(ValueError):
            opt.step(grads)
        own.pop()
    opt.master[0] = torch.zeros(40)
    with pytest.raises(ValueError):
        opt.step(grads)
    opt.master[0] = None
    opt.v[0] = opt.m[0]
    with pytest.raises(ValueError):
        opt.step(grads)
    assert not calls and opt.steps == 0


def test_parameters_stay(calls):
    opt, grads = optimizer(32)
    for change in (lambda p: p.__setitem__(0, torch.zeros(40)),
                   lambda p: p.append(torch.zeros(40)),
                   lambda p: p.__setitem__(0, None)):
        keep = list(opt.params)
        change(opt.params)
        with pytest.raises((ValueError, AttributeError)):
            opt.step(grads)
        opt.params[:] = keep
    opt.step(grads)
    assert len(calls) == 1


def test_the_memory_of_replaced_states_is_not_another_tensors(calls):
    """An address that the last step used is not given to other data while
    the step after it could take it for the state."""
    opt, grads = optimizer(32)
    opt.step(grads)
    at = opt.m[0].data_ptr()
    opt.m[0] = None
    for _ in range(8):
        t = torch.zeros(40)
        assert t.data_ptr() != at
        opt.m[0] = t
        opt.m[0] = None


def test_states_of_a_captured_step_stay(calls, monkeypatch):
    """A graph holds their addresses: nothing else may be stepped instead,
    and their memory is not given back."""
    opt = moe.AdamW([torch.zeros(40)], lr=1.0, device_steps=True)
    monkeypatch.setattr(optim_module, "_capturing", lambda device: True)
    # (replaced before the capture: what is captured)
    opt.v[0] = torch.zeros(40)
    opt.step([torch.zeros(40)])
    assert calls[0][0]["v"] == opt.v[0].data_ptr()
    monkeypatch.setattr(optim_module, "_capturing", lambda device: False)
    opt.step([torch.zeros(40)])
    at = opt.m[0].data_ptr()
    opt.m[0] = torch.zeros(40)
    with pytest.raises(ValueError, match="captured"):
        opt.step([torch.zeros(40)])
    assert at not in {torch.zeros(40).data_ptr() for _ in range(8)}
    assert len(calls) == 2


def test_a_replaced_schedule_is_checked(calls):
    """As the one that is given at first is: its address goes to the GPU."""
    opt = moe.AdamW([torch.zeros(40)], lr=1.0, lr_scale=torch.ones(1))
    for bad in (torch.ones(1, dtype=torch.float64), torch.ones(2), 0.5,
                torch.ones(1, device="meta"), torch.ones(())):
        opt.lr_scale = bad
        with pytest.raises((ValueError, AttributeError)):
            opt.step([torch.zeros(40)])
    assert not calls and opt.steps == 0
    opt.lr_scale = torch.ones(1)
    opt.step([torch.zeros(40)])
    opt.lr_scale = None
    opt.step([torch.zeros(40)])
    assert len(calls) == 2


def test_changing_types_and_missing_gradients(calls):
    opt, grads = optimizer(32)
    opt.step(grads)
    opt.step([None, grads[1].to(BF)])
    opt.step(grads)
    assert [[t["numel"] for t in c] for c in calls] == \
        [[40, 15], [0, 15], [40, 15]]
    assert [c[1]["grad_dtype"] for c in calls] == [0, 1, 0]
    assert [c[1]["param_dtype"] for c in calls] == [1, 1, 1]
    assert calls[-1][0]["grad"] == grads[0].data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("b2,steps", [(0.999, 4000), (0.95, 400)])
def test_second_moments_of_a_long_run(b2, steps):
    """8-bit second moments beside 32-bit ones of the same gradients.  The
    root's rounding is right in the mean, so v gains its variance.  With a = 1
    - b2, a code c and the root u^2 = b2 c^2 + a g^2 the variance is at most
    |u - c| s, s <= u / 8 the step, and |u - c| = a |g^2 - c^2| / (u + c):
    E c^2 <= E g^2 (1 + f / 8) / (1 - f / 8) with f = u / (u + c), and never
    less than E g^2.  f: |g| <= 6 c of 65536 values, u <= c sqrt(b2 + 36 a).
    The mean over the values is off by its sampling: a code is off by half a
    step or so, v by 2 / 16 of itself; six standard deviations."""
    n, g = 1 << 16, torch.Generator(device="cuda").manual_seed(9)
    # every place between two powers of two
    std = torch.exp2(torch.arange(n, device="cuda") // 32 / (n / 32))
    grad = torch.zeros(n, device="cuda")
    opts = [moe.AdamW([torch.zeros(n, device="cuda")], lr=0.0, betas=(0.9, b2),
                      state_bits=bits, seed=2) for bits in (32, 8)]
    for _ in range(steps):
        grad.normal_(generator=g).mul_(std)
        for opt in opts:
            opt.step([grad])
    full, codes = opts
    unit = torch.exp2(codes.v_scale[0].double() - 127).repeat_interleave(32)
    v = (codes.v[0].double() * unit) ** 2
    ratio = float((v / std ** 2).sum() / (full.v[0].double() / std ** 2).sum())
    far = (b2 + 36 * (1 - b2)) ** 0.5
    f = far / (1 + far)
    noise = 6 * 0.125 / n ** 0.5
    assert 1 - noise <= ratio <= (1 + f / 8) / (1 - f / 8) + noise, ratio


@pytest.mark.gpu
def test_a_replaced_state_outlives_the_steps_that_use_it():
    """Steps on a stream of their own: the memory of a state that was replaced
    is not another tensor's on the stream that it came from while they run."""
    n, side = 1 << 26, torch.cuda.Stream()
    p, grad = (torch.zeros(n, device="cuda") for _ in range(2))
    opt = moe.AdamW([p], lr=0.0)
    torch.cuda.synchronize()
    at = opt.m[0].data_ptr()
    done = torch.cuda.Event()
    with torch.cuda.stream(side):
        for _ in range(300):                 # (of 0.35 ms each)
            opt.step([grad])
        done.record()
        opt.m[0] = torch.zeros(n, device="cuda")
        opt.step([grad])
    # (not touched)
    other = [torch.empty(n, device="cuda") for _ in range(2)]
    places = {t.data_ptr() for t in other}
    running = not done.query()               # still, after the allocations
    assert at not in places or not running
    torch.cuda.synchronize()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_a_loaded_checkpoint(bits):
    """States put in others' place, and states copied into them: the same
    steps, bit for bit, and the replaced ones are left as they were."""
    g = torch.Generator(device="cuda").manual_seed(3)
    start = [torch.empty(n, device="cuda", dtype=BF).normal_(generator=g)
             for n in (70, 5000)]
    grads = [torch.empty(t.shape, device="cuda").normal_(generator=g)
             for t in start]

    def new():
        return moe.AdamW([t.clone() for t in start], lr=0.1, state_bits=bits,
                         master=True, seed=5)

    first = new()
    for _ in range(3):
        first.step(grads)
    names = lists(first)
    saved = {n: [t.clone() for t in getattr(first, n)] for n in names}
    copied, put = new(), new()
    for opt in (copied, put):
        opt.steps = 3
        for p, q in zip(opt.params, first.params):
            p.copy_(q)
    old = {n: list(getattr(put, n)) for n in names}
    before = {n: [t.clone() for t in old[n]] for n in names}
    for n in names:
        for t, s in zip(getattr(copied, n), saved[n]):
            t.copy_(s)
        setattr(put, n, [s.clone() for s in saved[n]])
    for opt in (first, copied, put):
        opt.step(grads)
    for opt in (copied, put):
        for n in ["params", *names]:
            for a, b in zip(getattr(first, n), getattr(opt, n)):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
    for n in names:
        for a, b in zip(before[n], old[n]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
