"""libfattn: exact, IO-aware tiled attention for B200 (sm_100a).

The compute path is the C-ABI library ``libfattn.so`` (CUDA kernels for
sm_100a); ``io_aware_exact_34_b200.fattn`` is its Python binding.  Import the
binding explicitly: it fails loudly when the library has not been built.
"""
import os
import sysconfig


def calls_path(torch_version: str) -> str:
    """Where the binding's native calls lie.  They are compiled against one torch and one Python, which their file is
    named after: with another of either there is no such file until the next build."""
    return os.path.join(os.path.dirname(os.path.abspath(__file__)),
                        f"_fattn_calls.torch-{torch_version}{sysconfig.get_config_var('EXT_SUFFIX')}")
