"""bench.py --optimizer, end to end: a step uploads its batch, not the
parameters that the optimizer has stepped."""
import types

import pytest

import bench

PARAMS = ("rab_pos", "rab_time", "w1", "w2")
BATCH = ("offsets", "num_targets", "num_contexts", "timestamps", "x", "dout")
OUT = ("out", "dx", "dw1", "dw2", "d_rab_pos", "d_rab_time")


@pytest.mark.parametrize("optimizer", [None, "adamw", "adamw8"])
def test_what_is_uploaded(optimizer):
    wl, pr = bench.LayerWorkload(), types.SimpleNamespace(**{n: n for n in PARAMS + BATCH + OUT})
    wl.optimizer = optimizer
    ins, outs = wl.host_io(pr)
    assert sorted(ins) == sorted(BATCH + (() if optimizer else PARAMS)) and sorted(outs) == sorted(OUT)


@pytest.mark.gpu
def test_steps_are_kept():
    """The bias tables, which AdamW steps in place, have moved by all of the run's steps: an element whose gradient keeps its
    sign moves by about lr (1e-4) at each of the first ones; one step cannot move it by more than 1.1 lr."""
    torch = pytest.importorskip("torch")
    from hstu_jagged_attention_02_gb300 import synth
    wl = bench.LayerWorkload()
    wl.optimizer = "adamw"
    b = synth.layer(5, n_lo=100, n_hi=300, B=3)
    pr = wl.problem(b, "cuda")
    opt = wl.make_optimizer(pr)
    before = pr.rab_pos.clone()
    args = types.SimpleNamespace(warmup=3, steps=5)
    e2e = bench.run_e2e(args, wl, [pr], [wl.flops(b)], torch.cuda.current_stream(), 1, opts=[opt])
    torch.cuda.synchronize()
    assert opt.steps() >= 8 and opt.device_error() == 0 and pr.device_error() == 0
    assert float((pr.rab_pos - before).abs().max()) > 3e-4
    assert torch.equal(pr.w1, opt.params[0].bfloat16()) and torch.equal(pr.w2, opt.params[1].bfloat16())
    assert e2e["h2d_bytes_per_step"] == sum(t.numel() * t.element_size() for t in wl.host_io(pr)[0])
