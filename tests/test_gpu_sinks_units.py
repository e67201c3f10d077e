"""The backward with sinks where its units are shared out in ways of their own: more
units with sinks than SMs, as many, and at d = 256 more clusters than run at once."""
import pytest
import torch

from flashattention_attention_backward_gb300.inputs import make_inputs
from oracle import attention_backward
from parity_helpers import check_grad
from test_gpu_sinks import _run, _w

pytestmark = pytest.mark.gpu


def _check(w, win, sinks):
    x = make_inputs(w)
    out = _run(w, win, sinks, x)
    f64 = [x[n].double().numpy() for n in ("q", "k", "v", "do")]
    grads = attention_backward(*f64, w.scale, w.causal, w.softcap, window=win, sinks=sinks)
    for name, g in zip(("dq", "dk", "dv"), grads):
        check_grad(name, out[name], g)


@pytest.mark.parametrize("w,win,sinks", [
    (_w(16, 8, 4, 600, 64, True), (20, -1), 300),        # 192 units with sinks of 320
    (_w(20, 4, 4, 500, 128, True, 5.0, 2.0), (70, -1), 500),  # nothing else
    (_w(41, 4, 4, 300, 64, False), (30, 10), 140),       # 328: more than two an SM
], ids=["192", "all", "328"])
def test_more_units_with_sinks_than_sms(w, win, sinks):
    _check(w, win, sinks)


def test_as_many_units_with_sinks_as_sms():
    """Every CTA takes one, and the others' units then come in snake order."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    _check(_w(sms, 1, 1, 300, 64, True), (20, -1), 4)


@pytest.mark.parametrize("w,win,sinks", [
    (_w(1, 2, 2, 2500, 256, True), (40, -1), 600),
    (_w(2, 4, 1, 1700, 256, True), (60, -1), 1100),
    (_w(3, 2, 1, 900, 256, False, 6.0, 2.0), (30, 20), 400),
], ids=["2500", "1700", "900"])
def test_more_clusters_than_run_at_once(w, win, sinks):
    _check(w, win, sinks)


@pytest.mark.parametrize("w,win,sinks", [
    (_w(1, 4, 2, 500, 128, False), (30, -1), 70),
    (_w(1, 2, 1, 700, 64, False, 4.0, 2.0), (0, -1), 200),
    (_w(1, 2, 2, 400, 256, False), (60, -1), 3),
], ids=["128", "64", "256"])
def test_no_right_bound(w, win, sinks):
    """Every key from the window's start on, and the first ones."""
    _check(w, win, sinks)
