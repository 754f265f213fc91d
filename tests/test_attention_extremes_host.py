"""Host checks of the attention operators at the ends of what they accept.  No GPU
needed."""
from test_attention_ops_host import (OK, SHAPE, _cached, _packed, _packed_grad, _status,  # noqa: F401
                                     lib)
from test_token_launches_host import launches  # noqa: F401  (a fixture)


def test_scales_whose_scores_are_no_numbers_in_units_of_log_2(lib, launches):  # noqa: F811
    """scale * log2(e) has to be a float32; what is refused launches nothing."""
    for make in (_packed, _packed_grad, _cached):
        for scale in (2.36e38, 2.4e38, 3.4e38):
            assert _status(lib, make(scale=scale)) == SHAPE, (make.__name__, scale)
        (status, made), = launches([[*make(scale=2.358e38), -1]])
        assert status == OK and made, make.__name__
