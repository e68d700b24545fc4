// The device error words of the translation units that cache_ops.cu reads along with its own.
#pragma once

namespace da {

int take_prefix_error_word(unsigned int* flags);
int take_sparse_error_word(unsigned int* flags);
int take_evict_error_word(unsigned int* flags);

}  // namespace da
