"""Calls at the edges of what the serving operators take: tensors in host memory among the device's."""
import pytest
import torch

from test_serving_checks import NAMES, calls

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def xv():
    from bit_exact_speculative_gb300 import build
    build.build()
    from bit_exact_speculative_gb300 import xv as m
    return m


def on_device(xv, name):
    args = {k: t.cuda() if torch.is_tensor(t) else t for k, t in calls(xv)[name].items()}
    if "pages" in args:
        args["pages"] = xv.kv_pages(args["pages"]._table.cuda(), args["pages"].page_size, args["pages"].n_pages)
    return args


@pytest.mark.parametrize("name", NAMES)
def test_one_tensor_in_host_memory_is_refused(xv, name):
    """Each tensor in turn, the first one among them (it says which device the others must be on)."""
    args = on_device(xv, name)
    for k, t in args.items():
        if torch.is_tensor(t):
            with pytest.raises(ValueError, match="device"):
                getattr(xv, name)(**dict(args, **{k: t.cpu()}))
    if "pages" in args:
        with pytest.raises(ValueError, match="page_table"):
            getattr(xv, name)(**dict(args, pages=xv.kv_pages(args["pages"]._table.cpu(), args["pages"].page_size, args["pages"].n_pages)))
    getattr(xv, name)(**args)      # the least sizes are enough
    getattr(xv, name)(**args, stream=torch.cuda.current_stream())
    assert xv.xv_device_check() == 0
