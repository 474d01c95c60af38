"""CPU oracle for token-level KV selection (test infrastructure only).

Only ``tests/``, ``__graft_entry__.smoke()`` and ``bench.py``'s CPU-baseline
and reference legs may import this package. The product path never calls it.
"""
from .tokenselect_oracle import *  # noqa: F401,F403
from .cache4_oracle import (attention, prompt_attention, q4_pack, q4_pool_values, q4_quantise,  # noqa: F401
                            q4_values, round_bf16)
