"""The workspace that the binding allocates when none is given."""
import pytest

from tests._attn import Batch, check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import gated_delta_ssm_gb300 as gdn  # noqa: E402

CALLS = {"decode": gdn.attn_decode, "prefill": gdn.attn_prefill}


def _streams_with_memory():
    return {s["stream"] for s in torch.cuda.memory_snapshot()}


def _unused_stream():
    torch.cuda.synchronize()
    used = _streams_with_memory()
    return next(s for s in (torch.cuda.Stream() for _ in range(64)) if s.cuda_stream not in used)


@pytest.mark.parametrize("form", ["decode", "prefill"])
@pytest.mark.parametrize("raw", [False, True])
def test_it_belongs_to_the_stream_of_the_call(form, raw):
    # memory of the current stream's pool may still be in use by work queued there, which the call's stream does not
    # wait for
    t = Batch([1, 2], [3000, 200], 8, 2, 64, seed=1)
    t.make_q()
    want, bound = t.expected(128 ** -0.5)
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    side = _unused_stream()
    CALLS[form](t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(),
                stream=side.cuda_stream if raw else side)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    torch.cuda.synchronize()
    assert side.cuda_stream in _streams_with_memory()
    check(out, want, bound)
    assert gdn.check_device() == 0
    torch.cuda.empty_cache()


def test_the_default_stream_by_its_raw_handle():
    t = Batch([1], [500], 4, 1, 64, seed=3)
    t.make_q()
    out = torch.full((t.N, t.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    before = _streams_with_memory()
    gdn.attn_decode(t.q, t.cache(), t.d["q_start"], t.d["kv_len"], out, t.dims(), stream=0)
    torch.cuda.synchronize()
    assert _streams_with_memory() == before
    check(out, *t.expected(128 ** -0.5))


def test_that_of_the_chunked_prefill_too():
    from gated_delta_ssm_gb300 import synth
    from tests._util import check_out, device_inputs, dims_of, params_of, run_oracle
    shape = synth.Shape(B=1, T=70, Hq=1, Hv=2, warm=True)
    inp = synth.make_inputs(shape, seed=2)
    dev = device_inputs(shape, inp)
    out = torch.empty(1, 70, 2, shape.d, device="cuda")
    side = _unused_stream()
    gdn.prefill_chunked(dev["state"], dev["hist"], dev["x"], dev["z"], dev["alpha"], dev["beta_logit"], params_of(dev),
                        out, dims_of(shape), 70, 64, stream=side)
    torch.cuda.synchronize()
    assert side.cuda_stream in _streams_with_memory()
    check_out(out.cpu().numpy(), run_oracle(shape, inp)["out"])
    torch.cuda.empty_cache()
