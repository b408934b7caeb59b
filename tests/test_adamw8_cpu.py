"""AdamW8's states that are not there are refused as AdamW's are."""
import pytest
import torch

import sgd_gradient_all_amd as ddl
from sgd_gradient_all_amd import _operators as ops
from test_operators_cpu import OnDevice

E_NULL = -1


@pytest.mark.parametrize("name", ["m", "v", "m_scale", "v_scale"])
def test_missing_states(name, monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    d = lambda *s, dtype=torch.float32: OnDevice(0, *s, dtype=dtype)  # noqa: E731
    a = ddl.AdamW8([(0, 300)])
    ok = dict(grad=d(300), m=d(300, dtype=torch.int8), v=d(300, dtype=torch.uint8), m_scale=d(2),
              v_scale=d(2), weights=[d(300)], lr=1.0)
    with pytest.raises(ddl.DDLError) as e:
        a.step(**{**ok, name: None})
    assert e.value.code == E_NULL
