"""The operators' conveniences on another stream than the current one: memory that they allocate, read and return is not
given to anyone else while a kernel still uses it."""
import pytest
import torch

import dense_tensor_core_persistent_gb300 as g
from dense_tensor_core_persistent_gb300 import build as gbuild

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
A_WHILE = 100_000_000  # clock cycles, some 50 ms
NAMES = ["rms_norm", "rms_norm_e4m3", "rms_norm_backward", "token_logprobs", "token_logprobs_backward", "glu_bf16",
         "glu_e4m3", "glu_bf16_backward"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gbuild.build()


def operator(name):
    """(a call, the tensors it takes)."""
    gen = torch.Generator(device=DEV).manual_seed(len(name))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)

    if name.startswith("rms_norm"):
        x, r, w = normal(2000, 1024), normal(2000, 1024), normal(1024)
        if name != "rms_norm_backward":
            out = "e4m3" if name.endswith("e4m3") else "bf16"
            return lambda x, w, r, stream=None: g.rms_norm(x, w, residual=r, out=out, save=True, stream=stream), [x, w, r]
        n = g.rms_norm(x, w, residual=r, save=True)
        return g.rms_norm_backward, [normal(2000, 1024), n.sum, w, n.rstd, r]
    if name.startswith("token"):
        l, t = normal(300, 8000), torch.arange(300, device=DEV)
        if name == "token_logprobs":
            return lambda l, t, stream=None: g.token_logprobs(l, t, top=4, stream=stream), [l, t]
        r = g.token_logprobs(l, t)
        return g.token_logprobs_backward, [l, t, r.lse, r.entropy, torch.ones(300, device=DEV)]
    x, wg, wu = normal(300, 512), normal(1024, 512), normal(1024, 512)
    if name == "glu_bf16":
        return lambda x, wg, wu, stream=None: g.glu_bf16(x, wg, wu, save=True, stream=stream), [x, wg, wu]
    if name == "glu_e4m3":
        one = torch.ones(1024, device=DEV)
        x, wg, wu = (t.to(torch.float8_e4m3fn) for t in (x, wg, wu))
        return g.glu_e4m3, [x, one[:300].clone(), wg, one, wu, one.clone()]
    _, saved = g.glu_bf16(x, wg, wu, save=True)
    return g.glu_bf16_backward, [normal(300, 1024), x, wg, wu, saved]


def tensors(got):
    return [got] if isinstance(got, torch.Tensor) else [t for t in got if t is not None]


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(tensors(a), tensors(b)))


def fill_the_like(ts):
    """Takes memory of the sizes of `ts` from the current stream and gives it back with writes still to come."""
    for t in [torch.empty_like(t) for t in ts for _ in range(2)]:
        bits(t).fill_(0xFF)


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_do_not_take_memory_that_the_current_stream_still_writes(name, handle):
    call, args = operator(name)
    want = call(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(A_WHILE)
    fill_the_like(tensors(want))
    got = call(*args, stream=side.cuda_stream if handle else side)
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_inputs_are_kept_until_the_other_stream_has_read_them(name):
    call, args = operator(name)
    want = call(*args)
    sizes = [torch.empty_like(t, device="meta") for t in args]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(A_WHILE)
    got = call(*args, stream=side)
    del args
    fill_the_like([torch.empty_like(t, device=DEV) for t in sizes])
    torch.cuda.synchronize()
    assert same(got, want)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_kept_until_the_current_stream_has_read_them(name):
    call, args = operator(name)
    want = call(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(A_WHILE)
    copies = [t.clone() for t in tensors(got)]
    del got
    with torch.cuda.stream(side):
        fill_the_like(copies)
    torch.cuda.synchronize()
    assert same(copies, want)


def test_the_current_stream_named_is_the_current_stream():
    call, args = operator("rms_norm")
    want = call(*args)
    got = call(*args, stream=torch.cuda.current_stream())
    again = call(*args, stream=torch.cuda.current_stream().cuda_stream)
    assert same(got, want) and same(again, want)
