// fake_products.cpp -- keeps what the tiled products' launches are given:
// shapes and how their items are dealt out.  fake_cudart.cpp is compiled with its
// launch renamed to fake_launch, which this one calls.
#include <cstring>

#include <cuda_runtime_api.h>

extern "C" cudaError_t fake_launch(const cudaLaunchConfig_t* c, const void* f, void** args);

namespace {

struct Product {  // of a launch
    int shapes[2][7];  // m, n, tiles of each, splits, chains, blocks; zero: none
    int deal[6];       // pairs, longs, ahead, shorts, after, before
};
constexpr int kMost = 4096;
Product products[kMost];
int count = 0;

}  // namespace

extern "C" {

void fake_products_clear(void) { count = 0; }
int fake_products(void) { return count; }
const int* fake_product(int i) { return products[i].shapes[0]; }

cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args)
{
    // only the products have so many threads and so much shared memory
    if (c->blockDim.x == 384 && c->dynamicSmemBytes > 128 * 1024 && count < kMost) {
        Product& p = products[count++];
        std::memcpy(p.shapes[0], args[2], sizeof p.shapes[0]);
        std::memcpy(p.shapes[1], args[6], sizeof p.shapes[1]);
        std::memcpy(p.deal, args[8], sizeof p.deal);
    }
    return fake_launch(c, f, args);
}

}  // extern "C"
