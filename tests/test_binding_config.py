"""The C structure that a call takes from a Config is that of the fields as they
are at the call, however they came to be."""
import pytest

import block_scaled_expert_amd as bse


def _top_k(cfg):
    return cfg.ref()._obj.top_k


def test_fields_set_past_setattr():
    cfg = bse.Config(top_k=4)
    assert _top_k(cfg) == 4
    vars(cfg)["top_k"] = 5
    assert _top_k(cfg) == 5
    cfg.__dict__.update(top_k=6)
    assert _top_k(cfg) == 6
    object.__setattr__(cfg, "top_k", 7)
    assert _top_k(cfg) == 7
    del cfg.top_k
    assert _top_k(cfg) == bse.Config.top_k
    cfg.top_k = 4
    assert _top_k(cfg) == 4 and cfg.ref()._obj.hidden == cfg.hidden


def test_values_that_change_in_place():
    import numpy as np
    scale = np.array(1.0, dtype=np.float32)
    cfg = bse.Config(fmt="nvfp4", act_gs=bse.ACT_GS_STATIC, act_gs_static=(scale, 1.0))
    assert cfg.ref()._obj.act_gs_static[0] == 1.0
    scale[...] = 2.0
    assert cfg.ref()._obj.act_gs_static[0] == 2.0

    import torch
    cap = torch.tensor(3.0)
    cfg = bse.Config(cap=cap)
    assert cfg.ref()._obj.cap == 3.0
    cap.fill_(4.0)
    assert cfg.ref()._obj.cap == 4.0


def test_a_subclass_has_its_own_structure():
    class Half(bse.Config):
        @property
        def num_local(self):
            return self.num_experts // 2

    class Other:
        __slots__ = ("more",)

    class Both(bse.Config, Other):
        pass

    a, b = bse.Config(), Half()
    assert a.ref()._obj.num_local_experts == a.num_experts and b.ref()._obj.num_local_experts == b.num_experts // 2
    assert Both(top_k=3).ref()._obj.top_k == 3


def test_a_field_set_while_the_structure_is_built():
    """As by another thread: what was read before is not kept for later calls."""
    class Name(str):
        """A format name that sets another field when it is looked up, at the
        second time: the structure takes top_k between the first and that."""
        def __hash__(self):
            seen.append(1)
            if len(seen) == 2:
                cfg.top_k = 5
            return str.__hash__(self)

    cfg = bse.Config(fmt=Name("nvfp4"), top_k=4, cap=1.2345)     # of no other test
    seen = []
    cfg.ref()
    assert len(seen) >= 2
    assert _top_k(cfg) == 5
    assert bse.Config(top_k=4).ref()._obj.top_k == 4


def test_equal_configs_of_many_values():
    for n in range(1, 300):
        cfg = bse.Config(top_k=n, cap=float(n))
        assert _top_k(cfg) == n and cfg.ref()._obj.cap == float(n)
    with pytest.raises(ValueError):
        bse.Config(fmt="fp4").ref()
